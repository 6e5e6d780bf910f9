"""Runs a fixed set of small 8-bit row, product and sampling calls through one
build of the library and saves every output:
`python tests/_checked_q8_cases.py LIB OUT.npz`. test_gpu_q8_checked.py runs it
once with libglance.so and once with the bounds-checked libglance_check.so and
compares the two. Inputs are seeded."""
import os
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))

import tree_verified_block_gb300._binding as b  # noqa: E402

b.LIB_PATH = sys.argv[1]

import torch  # noqa: E402

import tree_verified_block_gb300 as g  # noqa: E402


def main(out_path):
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    gen = torch.Generator(device=dev).manual_seed(12)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    res = {}
    for dtype in (torch.bfloat16, torch.float32):
        for M, d in ((1, 16), (5, 528), (130, 4096), (3, 16384)):
            x, r, w = rn(M, d).to(dtype), rn(M, d).to(dtype), 1 + 0.1 * rn(d)
            c, s, t, out = torch.zeros(M, d, dtype=torch.uint8, device=dev), torch.zeros(M, device=dev), torch.zeros_like(x), torch.zeros_like(x)
            g.q8_norm_rows(x, r, w, 1e-6, t, c, s)
            g.q8_read_rows(c, s, out)
            key = f"{M}_{d}_{dtype}"
            for n, v in (("codes", c), ("scales", s), ("total", t), ("back", out)):
                res[n + key] = v.float().cpu().numpy()
    for M, K, N, gated, dtype in ((1, 4096, 256, False, torch.bfloat16), (17, 1040, 136, True, torch.float32), (64, 512, 4096, False, torch.float32),
                                  (100, 256, 30000, False, torch.bfloat16), (200, 512, 520, True, torch.bfloat16), (300, 144, 264, False, torch.float32),
                                  (700, 512, 10008, True, torch.bfloat16)):
        x, xs, w, ws = (torch.zeros(n, K, dtype=torch.uint8, device=dev) if i % 2 == 0 else torch.zeros(n, device=dev)
                        for i, n in enumerate((M, M, N * (1 + gated), N * (1 + gated))))
        g.q8_rows(rn(*x.shape), x, xs)
        g.q8_rows(rn(*w.shape), w, ws)
        out = rn(M, N).to(dtype)
        g.q8_linear(x, xs, w, ws, out, bias=rn(w.shape[0]), act="silu", gated=gated, residual=out)
        res[f"linear{M}_{K}_{N}"] = out.float().cpu().numpy()
    for M, V in ((3, 2), (5, 1001), (7, 40000), (25, 20000)):
        for dtype in (torch.bfloat16, torch.float32):
            x = (2 * rn(M, V)).to(dtype)
            row = lambda *v: torch.tensor([v[i % len(v)] for i in range(M)], device=dev)
            tokens, gap = torch.zeros(M, dtype=torch.int32, device=dev), torch.zeros(M, device=dev)
            g.sample(x, row(0.7, 1.0, 0.0, 1.3), row(20, 0, 0, 5000, 700).int(), row(0.9, 0.5, 1.0), row(0.0, 0.0, 0.05), 7,
                     torch.arange(M, dtype=torch.int32, device=dev), None, tokens, gap)
            res[f"tokens{M}_{V}_{dtype}"], res[f"gap{M}_{V}_{dtype}"] = tokens.cpu().numpy(), gap.cpu().numpy()
    st = torch.zeros(g.STATUS_WORDS, dtype=torch.int32, device=dev)
    g.get_status(st)
    torch.cuda.synchronize()
    res["status"] = st.cpu().numpy()
    np.savez(out_path, **res)


if __name__ == "__main__":
    main(sys.argv[2])
