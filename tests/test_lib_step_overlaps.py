"""Calls of include/tq_step.h whose outputs meet an input or each other are refused before any launch (fake
pointers, no GPU)."""

import os

import pytest

import rotation_lloyd_max_amd as tq
from rotation_lloyd_max_amd import step
from test_lib_kv_host import ERR_ARG, cache

pytestmark = pytest.mark.skipif(not os.path.exists(tq.LIB_PATH), reason="libtq.so not built")

KB = 1 << 20
B, M, PAGES, WIDTH, WORDS, V = 3, 7, 4, 10, 2, 100
ROWS = PAGES * 8 * 64        # of a half of the cache: pages, heads, tokens of a page
# arrays of a call and their bytes, each at a place of its own
PLAN = dict(lens=4 * B, counts=4 * B, page_table=4 * B * WIDTH, parents=4 * M, shift=4 * B, slots=8 * M, positions=4 * M,
            q_offsets=4 * B + 4, kv_lens=4 * B, status=4 * B, tree=4 * M * WORDS, left=4, free=4 * PAGES, state=8)
KEEP = dict(lens=4 * B, q_offsets=4 * B + 4, status=4 * B, kept=4 * B, path=4 * M, page_table=4 * B * WIDTH, lens_out=4 * B, left=4,
            free=4 * PAGES, state=8, k_codes=ROWS * 128, k_scales=ROWS * 2 * 128 // 64, v_codes=ROWS * 48, v_scales=ROWS * 2 * 128 // 64)
VERIFY = dict(target=2 * V * M, draft=2 * V * M, offsets=4 * B + 4, tokens=4 * M, parents=4 * M, uniforms=4 * M, temperature=4 * B,
              kept=4 * B, out_tokens=4 * M, path=4 * M, ws=256)
WRITTEN = dict(plan={"page_table", "slots", "positions", "q_offsets", "kv_lens", "status", "tree", "left", "state"},
               keep={"lens_out", "left", "free", "state", "k_codes", "k_scales", "v_codes", "v_scales"}, verify={"kept", "out_tokens", "path", "ws"})


def places(sizes):
    return {n: (i + 1) * KB for i, n in enumerate(sizes)}


def plan(a):
    p = step._KVPool(a["free"], a["state"], PAGES)
    return tq.lib().tq_kv_plan(p, 64, B, a["lens"], a["counts"], a["page_table"], WIDTH, M, a["parents"], a["shift"], a["slots"],
                               a["positions"], a["q_offsets"], a["kv_lens"], a["status"], a["tree"], WORDS, a["left"], None)


def keep(a):
    p = step._KVPool(a["free"], a["state"], PAGES)
    c = cache(k=dict(codes=a["k_codes"], scales=a["k_scales"]), v=dict(codes=a["v_codes"], scales=a["v_scales"]))
    return tq.lib().tq_kv_keep(p, c, 64, B, a["lens"], a["q_offsets"], a["status"], a["kept"], a["path"], M,
                               a["page_table"], WIDTH, a["lens_out"], a["left"], None)


def verify(a, stride=V):
    return tq.lib().tq_verify(a["target"], tq.BF16, stride, a["draft"], tq.BF16, stride, 0, V, B, a["offsets"], M, a["tokens"],
                              a["parents"], a["uniforms"], a["temperature"], a["kept"], a["out_tokens"], a["path"], a["ws"],
                              1 << 19, None)


CALLS = dict(plan=(plan, PLAN), keep=(keep, KEEP), verify=(verify, VERIFY))
PAIRS = [(call, w, o) for call, (_, sizes) in CALLS.items() for w in sorted(WRITTEN[call]) for o in sizes if o != w]


@pytest.mark.parametrize("call,written,other", PAIRS)
def test_an_output_that_meets_another_array(call, written, other):
    fn, sizes = CALLS[call]
    for end in (False, True):
        a = places(sizes)
        if written == "ws":      # (256-byte aligned, so the other one is moved)
            a[other] = a["ws"] + (192 if end else 0)
        else:                    # at its start, or with the first element in the other's last
            a[written] = a[other] + (sizes[other] - 8 if end and sizes[other] > 8 else 0)
            if written == "slots" or written[:2] in ("k_", "v_"):       # (aligned as they have to be)
                a[written] &= ~15
        same = call == "keep" and {written, other} == {"lens", "lens_out"} and a["lens"] == a["lens_out"]
        taken = {written, other} == {"left", "state"} and a["left"] == a["state"]
        if same or taken:
            continue             # (in place; the pages are taken)
        assert fn(a) == ERR_ARG, (call, written, other)
        assert b"overlap" in tq.lib().tq_last_error()


def test_a_row_of_a_distribution_far_behind_the_first():
    a = places(VERIFY)
    a["target"], a["draft"] = 32 * KB, 64 * KB
    for name in ("kept", "out_tokens", "path"):
        for row in (0, 3, M - 1):
            assert verify({**a, name: a["target"] + row * KB + 2 * V - 4}, KB // 2) == ERR_ARG
            assert b"overlap" in tq.lib().tq_last_error()
