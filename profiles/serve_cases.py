"""The programs behind serve_kernels.md: position rotation, block tables, verification and drawing.

    python profiles/serve_cases.py rope|blocks|verify|draw
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import turboquant_compressed_kv_tq_gb300 as tq  # noqa: E402


def rope():
    qkv = torch.randn(1, 8192, 80, 128, device="cuda").to(torch.bfloat16).transpose(1, 2)
    r, starts = tq.Rope.of_base(128), torch.full((1,), 253952, dtype=torch.int32, device="cuda")
    out, k_out = r.apply(qkv[:, :64], qkv[:, 64:72], starts=starts)
    return lambda: r.apply(qkv[:, :64], qkv[:, 64:72], out, k_out, starts=starts)


def blocks():
    B, n = 512, 2048
    bt, lens = tq.BlockTable(B, 64, B * 64, 64), torch.zeros(B, dtype=torch.int32, device="cuda")
    places = tq.Places(B, B * n)

    def run():
        bt.reserve(lens, None, n, places)
        bt.release(lens)
    return run


def verify():
    B, K, V = 64, 4, 131072
    common = 4 * torch.randn(B, K + 1, V, device="cuda")
    q = torch.softmax(common[:, :K] + 1.5 * torch.randn(B, K, V, device="cuda"), -1)
    x = (common + 1.5 * torch.randn_like(common)).to(torch.bfloat16)
    drafts = (q / torch.empty_like(q).exponential_()).argmax(-1).to(torch.int32)
    u, e = torch.rand(B, K, device="cuda"), torch.empty(B, V, device="cuda").exponential_()
    return lambda: tq.tq_verify_drafts(x, drafts, q, u, e)


def draw():
    B, V = 200, 131072
    x, e = 4 * torch.randn(B, 1, V, device="cuda"), torch.empty(B, V, device="cuda").exponential_()
    return lambda: tq.tq_verify_drafts(x, noise=e)


if __name__ == "__main__":
    torch.manual_seed(0)
    run = {"rope": rope, "blocks": blocks, "verify": verify, "draw": draw}[sys.argv[1]]()
    for _ in range(3):
        run()
    torch.cuda.synchronize()
    assert tq.tq_device_error() == 0
