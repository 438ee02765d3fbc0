"""Calls around the caches' whose outputs share memory with what they read, or with each other: host only."""
import ctypes

import pytest
import torch

import turboquant_compressed_kv_tq_gb300 as tq  # noqa: F401
from test_serve_refusals import INVALID, lib  # noqa: F401 (lib: fixture)
from turboquant_compressed_kv_tq_gb300 import _lib

# addresses that are never looked at
B, K, V, S = 3, 2, 100, 1 << 16
AT = {name: (i + 1) << 20 for i, name in enumerate(
    ["target", "draft", "draft_tokens", "draft_lens", "temperatures", "uniforms", "noise", "seq_lens", "accepted", "tokens", "logprobs", "keep_lens"])}
BYTES = {"target": B * (K + 1) * V * 2, "draft": B * K * V * 4, "draft_tokens": 4 * B * K, "draft_lens": 4 * B, "temperatures": 4 * B, "uniforms": 4 * B * K,
         "noise": B * V * 4, "seq_lens": 4 * B, "accepted": 4 * B, "tokens": 4 * B * (K + 1), "logprobs": 4 * B * (K + 1), "keep_lens": 4 * B}
OUT = ["accepted", "tokens", "logprobs", "keep_lens"]


def verify(lib, noise=True, **at):
    a = AT | at
    d = _lib.tq_drafts(a["target"], (K + 1) * V, V, a["draft"], K * V, V, a["draft_tokens"], a["draft_lens"], a["temperatures"], a["uniforms"],
                       a["noise"] if noise else None, V, a["seq_lens"], 1, 0, 0)
    return lib.tq_verify_drafts(ctypes.addressof(d), B, K, V, a["accepted"], a["tokens"], a["logprobs"], a["keep_lens"], None)


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("other", list(AT))
def test_outputs_of_a_verification(lib, out, other):  # noqa: F811
    if out == other:
        return
    where = {AT[other], AT[other] + BYTES[other] - 4, AT[other] + BYTES[other] // 8 * 4, AT[other] - BYTES[out] + 4}
    if (out, other) == ("keep_lens", "seq_lens"):
        where.remove(AT[other])
    for at in where:
        assert verify(lib, **{out: at}) == INVALID, at
    assert verify(lib, keep_lens=AT["seq_lens"], **({out: AT["seq_lens"]} if out != "keep_lens" else {"accepted": AT["seq_lens"]})) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="these calls pass the checks, and nothing is at their addresses")
def test_verifications_that_share_nothing(lib):  # noqa: F811
    passed = _lib.TQ_ERR_CUDA   # (no device)
    assert verify(lib) == passed
    assert verify(lib, keep_lens=AT["seq_lens"]) == passed
    for out in OUT:
        for other in AT:
            if out != other:
                assert verify(lib, **{out: AT[other] + BYTES[other]}) == passed and verify(lib, **{out: AT[other] - BYTES[out]}) == passed
    # what a greedy call does not look at
    assert verify(lib, noise=False, logprobs=AT["uniforms"], accepted=AT["temperatures"], tokens=AT["draft"]) == passed


ROWS, WIDTH, FREE, MOST = 3, 4, 9, 12
BLOCKS = ["table", "free_blocks", "n_used", "granted", "starts", "seq_ids", "positions", "slots", "lens", "news"]
BLOCKS_AT = {name: (i + 1) << 20 for i, name in enumerate(BLOCKS)}
BLOCKS_BYTES = {"table": 4 * ROWS * WIDTH, "free_blocks": 4 * FREE, "n_used": 4, "granted": 4 * ROWS, "starts": 4 * ROWS + 4, "seq_ids": 4 * MOST, "positions": 4 * MOST,
                "slots": 8 * MOST, "lens": 4 * ROWS, "news": 4 * ROWS}


def reserve(lib, release=False, **at):
    a = BLOCKS_AT | at
    b = _lib.tq_blocks(a["table"], a["free_blocks"], a["n_used"], FREE, WIDTH, 16, FREE)
    p = _lib.tq_places(a["granted"], a["starts"], a["seq_ids"], a["positions"], a["slots"], MOST)
    if release:
        return lib.tq_blocks_release(ctypes.addressof(b), ROWS, a["lens"], None)
    return lib.tq_blocks_reserve(ctypes.addressof(b), ROWS, a["lens"], a["news"], 4, ctypes.addressof(p), None)


@pytest.mark.parametrize("out", BLOCKS[:8])
@pytest.mark.parametrize("other", BLOCKS)
def test_outputs_of_a_reservation(lib, out, other):  # noqa: F811
    if out == other:
        return
    where = {BLOCKS_AT[other], BLOCKS_AT[other] + BLOCKS_BYTES[other] - 4, BLOCKS_AT[other] - BLOCKS_BYTES[out] + 4}
    if (out, other) == ("granted", "news"):
        where.remove(BLOCKS_AT[other])
    for at in where:
        assert reserve(lib, **{out: at}) == INVALID
        if {out, other} <= {"table", "free_blocks", "n_used", "lens"}:
            assert reserve(lib, release=True, **{out: at}) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="these calls pass the checks, and nothing is at their addresses")
def test_reservations_that_share_nothing(lib):  # noqa: F811
    passed = _lib.TQ_ERR_CUDA   # (no device)
    assert reserve(lib) == passed and reserve(lib, release=True) == passed
    assert reserve(lib, granted=BLOCKS_AT["news"]) == passed and reserve(lib, lens=BLOCKS_AT["news"]) == passed
    for out in BLOCKS[:8]:
        for other in BLOCKS:
            if out != other:
                assert reserve(lib, **{out: BLOCKS_AT[other] + BLOCKS_BYTES[other]}) == passed
                assert reserve(lib, **{out: BLOCKS_AT[other] - BLOCKS_BYTES[out]}) == passed
