"""Seeded runs of the operators around the step, for comparing the release and debug libraries.

Run as a script (``python tests/debug_operator_cases.py OUT.npz``) under the
library that MA_LIBRARY selects; tests/test_gpu_debug_operators.py runs it once
per library and compares. The cases reach every kernel whose device indexing
the debug build guards: the norm (small sets, the streaming ring, ragged edges)
and in-place clipping, the clipped AdamW and momentum passes, the lookup, both
sorts, the sums (vectors of 8, 2 and 1 columns, short and long runs), the zeros,
the partial rows, the largest logits and the weight scaling.
"""
import sys

import numpy as np
import torch

import adamw_hybrid_optimizer_muon_b200 as ma


def run(path):
    torch.cuda.set_device(0)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    res = {"debug_build": np.array(int(ma.ma_debug_build()))}

    def keep(name, *tensors):
        torch.cuda.synchronize()
        res[name + "_status"] = np.array(ma.ma_device_status())
        for i, t in enumerate(tensors):
            res[f"{name}_{i}"] = t.float().cpu().numpy()

    for k, sizes in enumerate([[1, 1280, 77], [8192 * 3 + 5, 100, 40001], [50] * 700]):
        grads = [(new(n + 3) * 1e-2).to((torch.float32, torch.bfloat16)[i % 2])[i % 3:n + i % 3] for i, n in enumerate(sizes)]
        clip = ma.GradClip(grads)
        clip.norm(max_norm=0.1)
        P, M, W = ([new(x.numel()) for x in grads[::2]] for _ in range(3))
        ma.adamw_step_fused(P, grads[::2], M, [w.square() for w in W], ma.adamw_hparams(step=2), clip=clip.buffer)
        clip.clip(0.1, scale=2.0)
        keep(f"clip{k}", clip.buffer[:4], *grads[:20], *P[:20], *M[:20])
    for k, shape in enumerate([(256, 384), (384, 256)]):
        hp = ma.muon_hparams()
        Wt, Mo, Gr = [new(*shape)], [new(*shape) * 1e-3], [(new(*shape) * 1e-2).bfloat16()]
        clip = ma.GradClip(Gr)
        clip.norm(max_norm=0.1)
        ws = torch.empty(ma.muon_workspace_bytes(1, *shape, hp), dtype=torch.uint8, device="cuda")
        ma.muon_step_batched(Wt, Gr, Mo, hp, ws, clip=clip.buffer)
        keep(f"muon{k}", Wt[0], Mo[0])
    r = np.random.default_rng(4)
    for k, (n, V, D, dt) in enumerate([(300, 50, 24, torch.float32), (5000, 700, 66, torch.bfloat16),
                                       (20000, 3000, 40, torch.bfloat16), (9000, 40, 7, torch.float32),
                                       (12000, 300000, 8, torch.bfloat16)]):
        ids = torch.from_numpy((V * r.random(n) ** 3).astype(np.int64)).cuda()
        dy, table = new(n, D).to(dt), new(V, D).to(dt)
        grad = torch.empty((V, D), dtype=dt, device="cuda")
        ma.embedding_grad(ids, dy, grad, scale=2.0)
        acc = table.clone()
        ma.embedding_grad(ids, dy, acc, accumulate=True)
        keep(f"embed{k}", grad[:2000], acc[:2000], ma.embedding_lookup(ids[:500], table, scale=3.0))
    for k, (S, T, H, KV, D) in enumerate([(2, 300, 4, 2, 64), (1, 700, 2, 2, 128), (3, 129, 2, 1, 256)]):
        q, kk = new(S, T, H, D).bfloat16(), new(S, T, KV, D).bfloat16()
        top = ma.qk_max_logit(q, kk)
        wq, wk = new(H * D, 33), new(KV * D, 33)
        ma.qk_clip(wq, wk, top, tau=2.0, kv_heads=KV)
        off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
        keep(f"qk{k}", top, wq, wk, ma.qk_max_logit(q[0], kk[0], causal=False, absolute=True, offsets=off))
    np.savez(path, **res)


if __name__ == "__main__":
    run(sys.argv[1])
