"""Host-side decisions of the feed-forward operators at unusual sizes, with no
GPU: seen through the workspace sizes, which differ between the ways that a
call may take."""
import ctypes
import os
import re

import pytest

import moe_expert_routing_amd as M
from moe_expert_routing_amd import ffn

P = 0x10000  # a pointer that nothing here dereferences


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    return M.lib()


def mat(rows, cols, mats=1, p=P, ld=None):
    ld = cols if ld is None else ld
    return ffn.Matrix(p, ld, rows * ld if mats > 1 else 0)


def rows_of(rows, experts, tile, top_k=2, entry=P):
    return ffn.ExpertRows(P, P, P, entry, rows, experts, tile, top_k)


def a256(nbytes):
    return (nbytes + 255) // 256 * 256


def up8(n):
    return (n + 7) // 8 * 8


def expert_gated(tokens, hidden, inter, rows, experts, tile, backward=False, grads=("dx", "dw"),
                 x=None):
    w = mat(inter, hidden, experts)
    none = ffn.Matrix()
    return ffn.GatedFfnArgs(
        0, 1, tokens, hidden, inter, rows_of(rows, experts, tile),
        x or mat(tokens, hidden), w, w, mat(rows, inter), mat(rows, 2 * inter),
        mat(rows, inter) if backward else none,
        mat(rows, hidden) if backward and "dx" in grads else none,
        *([w, w] if backward and "dw" in grads else [none, none]))


# tokens, hidden, where the row of a token can lie past 4 GB in what the product reads:
# x itself, or the copy of it with its rows padded to 8 elements
WIDE = [
    (2_130_000, 1001, False), (2_131_000, 1001, True), (2_140_000, 1001, True),
    (2_146_000, 1001, True), (1_048_000, 2047, False), (1_049_000, 2047, True),
    (30_000_000, 65, True), (299_500, 7161, False), (299_700, 7161, True), (299_700, 7160, False),
]


@pytest.mark.parametrize("tokens,hidden,wide", WIDE)
def test_gathered_rows_of_a_copy_beyond_32_bits(L, tokens, hidden, wide):
    """Where a padded copy of x would be past what 32-bit offsets reach, the rows
    are gathered first: rows x width of workspace, not tokens x width."""
    rows, n, inter, tile = 4096, 8, 64, 256
    h8 = up8(hidden)
    weights = 0 if hidden == h8 else 2 * a256(n * inter * h8 * 2)
    x = a256((rows if wide else tokens) * h8 * 2) if wide or hidden != h8 else 0
    a = expert_gated(tokens, hidden, inter, rows, n, tile)
    assert L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 0) == x + weights
    dz = a256(rows * 2 * inter * 2)
    a = expert_gated(tokens, hidden, inter, rows, n, tile, True, ("dw",))
    assert L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 1) == dz + x


def test_misaligned_x_counts_as_its_copy(L):
    """x a few elements off the 16-byte grid, contiguous: 4 GB is its copy's size."""
    tokens, rows, n = 2_131_000, 4096, 8
    for hidden, wide in ((1004, True), (1001, True), (992, False)):
        h8 = up8(hidden)
        a = expert_gated(tokens, hidden, 64, rows, n, 256, x=mat(tokens, hidden, p=P + 2))
        weights = 0 if hidden == h8 else 2 * a256(n * 64 * h8 * 2)
        assert L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 0) == \
            a256((rows if wide else tokens) * h8 * 2) + weights


def test_the_headers_envelope_is_the_codes(L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moe_ffn.h")).read()
    most = 1 << int(re.search(r"#define MOE_FFN_MAX_ROWS \(1 << (\d+)\)", text).group(1))
    assert re.search(r"tokens and rows up to 2\^%d\b" % (most.bit_length() - 1), text)

    def linear(rows, experts=0):
        w = mat(64, 64, max(1, experts))
        none = ffn.Matrix()
        desc = rows_of(rows, experts, 16) if experts else ffn.ExpertRows()
        return ffn.LinearArgs(0, 0, rows, 64, 64, desc, mat(rows, 64), w, none, none, mat(rows, 64),
                              none, none, none, none, none)
    for experts in (0, 4):
        size = [L.moe_linear_workspace_bytes(ctypes.byref(linear(n, experts)), 0)
                for n in (most, most + 1)]
        assert size[0] >= 0 and size[1] == -1
    for kw in (dict(tokens=most + 1, rows=1), dict(tokens=1, rows=most + 1)):
        y = mat(1, 64)
        a = ffn.CombineArgs(0, 64, kw["tokens"], kw["rows"], 1, 4, 8, P, P, P, P, P, P, P, y, y, y,
                            y, y, P)
        assert L.moe_combine(ctypes.byref(a), None) == -4
        assert L.moe_combine_backward(ctypes.byref(a), None) == -4


# experts, tile, rows of the layout: whether its experts may be taken to have few rows. The
# few-row products read odd widths in place, the tiles read padded copies.
FEW = [
    (64, 256, 4096, False),     # exact, two experts with 2000 rows each
    (64, 256, 16384, False),    # every expert half a tile on average
    (64, 4096, 4096, False),    # one expert with up to 4096
    (64, 16, 1024, True),       # decode: a tile an expert
    (112, 16, 1776, True),      # the same with buffers of fixed size
    (112, 16, 96, True),        # a few of the experts
]


@pytest.mark.parametrize("experts,tile,rows,few", FEW)
def test_experts_without_entries_have_no_padding(L, experts, tile, rows, few):
    """At most rows / tile experts have rows, and only those have padding to take off
    the estimate of what an expert has."""
    H, F = 1001, 64
    a = expert_gated(5000, H, F, rows, experts, tile)
    got = L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 0)
    assert (got == 0) == few
    a = expert_gated(5000, H, F, rows, experts, tile, True, ("dw",))
    got = L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 1)
    assert (got < a256(5000 * up8(H) * 2)) == few


@pytest.mark.parametrize("rows,experts", [(8, 0), (1, 0), (1024, 64)])
def test_weight_gradients_of_few_rows_need_no_workspace(L, rows, experts):
    """They are made from dh and pre; the pre-activations' gradient is for dx alone."""
    H, F = 1001, 72
    a = expert_gated(rows, H, F, rows, max(1, experts), 16, True, ("dw",))
    if not experts:
        a.rows = ffn.ExpertRows()
    assert L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 1) == 0
    a.dx = mat(rows, H)
    assert L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 1) >= rows * 2 * F * 2
