"""The programs behind kv8_kernels.md: one layer's append, decode and prompt over the 8-bit cache.

    python profiles/kv8_cases.py append|decode|prompt
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import turboquant_compressed_kv_tq_gb300 as tq  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def main(what):
    D, H, G = 128, 8, 4
    B, N, BT, L = {"append": (1, 8192, 64, 1), "decode": (8, 16384, 16, 1), "prompt": (1, 8192, 256, 2048)}[what]
    width = N // BT + 1
    torch.manual_seed(0)
    c = tq.KV8Cache(1, B * width, BT, H, D)
    table = torch.randperm(B * width, device="cuda").to(torch.int32).view(B, width)
    rope = tq.Rope.of_base(D)
    k, v = (torch.randn(B, N, H, D, device="cuda").to(torch.bfloat16).transpose(1, 2) for _ in "kv")
    q = torch.randn(B, L, H * G, D, device="cuda").to(torch.bfloat16).transpose(1, 2)
    zero, n = i32([0] * B), i32([N] * B)
    out = torch.empty_like(q)
    ws = torch.empty(max(1, c.workspace_bytes(B, H * G, L, N)), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        c.append(0, k, v, zero, table, width, rope=rope)
        if what != "append":
            c.attention(0, q, n, table, width, N, out=out, workspace=ws, rope=rope)
    torch.cuda.synchronize()
    assert tq.tq_device_error() == 0


if __name__ == "__main__":
    main(sys.argv[1])
