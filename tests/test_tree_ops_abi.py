"""Refusals and size queries of the operators around drafted trees, pages and rotary positions: host
code only, no call here passes validation."""
import os
import random
import re

import pytest

w4 = pytest.importorskip("w4a16_mixed_precision_offline_amd")

A, B, MIS = 256, 512, 258  # fake addresses: aligned, misaligned
NULL, SHAPE, ALIGN, ARG = -1, -2, -3, -8


def refused(fn, code, *args):
    with pytest.raises(w4.W4A16Error) as e:
        fn(*args, stream=0)
    assert e.value.code == code, args


TREE = dict(parent=A, rows=A, lens=A, mask=A, depth=A, pos=A, batch=2, tokens=40, max_new=33, words=2, window=0)
LAYOUT = dict(kv_heads=1, head=128, group=64, page=64, pages=8, width=4)
ATTEND = dict(q=A, rows=A, lens=A, table=A, cache=A, mask=A, depth=A, out=A, lse=A, batch=2, tokens=40, max_new=33, max_len=100, words=2,
              ldq=512, ldo=512, q_heads=4, **LAYOUT, window=0, scale=0.1, dtype=0)
COMPACT = dict(cache=A, path=A, count=A, rows=A, lens=A, table=A, lens_out=B, batch=2, tokens=4, max_new=2, max_path=2, layers=2,
               layer_bytes=8 * 9216, **LAYOUT)
FORK = dict(cache=A, table=A, lens=A, parent=A, keep=A, room=A, pinned=A, table_out=B, lens_out=B, missing=A, batch=2, batch_out=3,
            layers=2, layer_bytes=8 * 9216, **LAYOUT)
ROTARY = dict(q=A, k=A, pos=A, axis=A, freq=A, qo=A, ko=A, tokens=4, q_heads=4, kv_heads=2, head=64, rot=64, axes=2, ldpos=4, ldq=256,
              ldk=128, ldqo=256, ldko=128, pairs=0, dtype=0)
BAD_LAYOUT = [
    (SHAPE, dict(kv_heads=0)), (SHAPE, dict(head=96)), (SHAPE, dict(group=16)), (SHAPE, dict(group=256)), (SHAPE, dict(head=64, group=128)),
    (SHAPE, dict(page=48)), (SHAPE, dict(page=0)), (SHAPE, dict(pages=0)), (SHAPE, dict(width=0)), (SHAPE, dict(width=1 << 25)),
    (SHAPE, dict(batch=0)), (SHAPE, dict(batch=65536)), (NULL, dict(cache=None)), (ALIGN, dict(cache=MIS)), (NULL, dict(table=None)),
    (NULL, dict(lens=None)), (ALIGN, dict(table=MIS)), (ALIGN, dict(lens=MIS))]
BAD_ROWS = [(NULL, dict(rows=None)), (ALIGN, dict(rows=MIS)), (SHAPE, dict(tokens=0)), (SHAPE, dict(max_new=0))]
BAD_LAYERS = [(SHAPE, dict(layers=0)), (SHAPE, dict(layers=(1 << 20) + 1)), (SHAPE, dict(layer_bytes=8 * 9216 - 16)),
              (SHAPE, dict(layer_bytes=8 * 9216 + 8)), (SHAPE, dict(layer_bytes=(1 << 46) + 16))]


@pytest.mark.parametrize("code,change", BAD_ROWS + [
    *[(NULL, {n: None}) for n in ("parent", "lens", "mask")],
    *[(ALIGN, {n: MIS}) for n in ("parent", "lens", "mask", "depth", "pos")],
    (SHAPE, dict(batch=0)), (SHAPE, dict(batch=65536)), (SHAPE, dict(max_new=41)), (SHAPE, dict(tokens=5000, max_new=4097, words=200)),
    (SHAPE, dict(words=1)), (SHAPE, dict(words=0)), (SHAPE, dict(window=-1))])
def test_tree_refusals(code, change):
    refused(w4.w4a16_kv4_tree, code, *{**TREE, **change}.values())


@pytest.mark.parametrize("code,change", BAD_LAYOUT + BAD_ROWS + [
    *[(NULL, {n: None}) for n in ("q", "out", "mask")], (NULL, dict(depth=None, window=3)),
    *[(ALIGN, {n: MIS}) for n in ("q", "out", "lse", "mask", "depth")],
    (SHAPE, dict(words=1)), (SHAPE, dict(words=0)), (SHAPE, dict(max_new=41)), (SHAPE, dict(ldq=504)), (SHAPE, dict(ldo=516)),
    (SHAPE, dict(q_heads=0)), (SHAPE, dict(q_heads=5, kv_heads=2)), (SHAPE, dict(max_len=0)), (SHAPE, dict(max_len=(1 << 30) + 1)),
    (SHAPE, dict(batch=4097, kv_heads=16384, q_heads=16384, ldq=1 << 21, ldo=1 << 21)),
    (SHAPE, dict(batch=1024, tokens=1 << 20, max_new=1 << 19, words=1 << 14)),
    (SHAPE, dict(window=-1)), (ARG, dict(scale=0.0)), (ARG, dict(scale=float("nan"))), (ARG, dict(dtype=2))])
def test_tree_attention_refusals(code, change):
    refused(w4.w4a16_kv4_tree_attention, code, *{**ATTEND, **change}.values())


@pytest.mark.parametrize("code,change", BAD_LAYOUT + BAD_ROWS + BAD_LAYERS + [
    *[(NULL, {n: None}) for n in ("path", "count", "lens_out")], *[(ALIGN, {n: MIS}) for n in ("path", "count", "lens_out")],
    (SHAPE, dict(max_path=0)), (SHAPE, dict(max_new=5)), (ARG, dict(lens_out=A))])
def test_compact_refusals(code, change):
    refused(w4.w4a16_kv4_compact, code, *{**COMPACT, **change}.values())


@pytest.mark.parametrize("code,change", BAD_LAYOUT + BAD_LAYERS + [
    *[(NULL, {n: None}) for n in ("parent", "table_out", "lens_out")],
    *[(ALIGN, {n: MIS}) for n in ("parent", "keep", "room", "table_out", "lens_out", "missing")],
    (SHAPE, dict(batch_out=0)), (SHAPE, dict(batch_out=2049)), (SHAPE, dict(pages=(1 << 19) + 1, layers=1)),
    (ARG, dict(table_out=A)), (ARG, dict(lens_out=A))])
def test_fork_refusals(code, change):
    refused(w4.w4a16_kv4_fork, code, *{**FORK, **change}.values())


@pytest.mark.parametrize("code,change", [
    *[(NULL, {n: None}) for n in ("q", "k", "pos", "freq", "qo", "ko", "axis")], *[(ALIGN, {n: MIS}) for n in ("q", "k", "pos", "axis", "freq")],
    (ALIGN, dict(q=264, qo=264)), (ALIGN, dict(ko=264)),
    (SHAPE, dict(tokens=0)), (SHAPE, dict(tokens=1 << 24, ldpos=1 << 26)), (SHAPE, dict(q_heads=0)), (SHAPE, dict(kv_heads=-1)),
    (SHAPE, dict(head=8, rot=8)), (SHAPE, dict(head=60, rot=48)), (SHAPE, dict(head=520)), (SHAPE, dict(rot=0)), (SHAPE, dict(rot=8)),
    (SHAPE, dict(rot=40)), (SHAPE, dict(rot=80)), (SHAPE, dict(axes=0)), (SHAPE, dict(ldpos=3)), (SHAPE, dict(ldq=248)),
    (SHAPE, dict(ldq=260, ldqo=260)), (SHAPE, dict(ldk=120)), (SHAPE, dict(ldqo=264)), (SHAPE, dict(ldko=136)),
    (SHAPE, dict(q_heads=1 << 19, ldq=1 << 25, ldqo=1 << 25)), (ARG, dict(pairs=2)), (ARG, dict(pairs=-1)), (ARG, dict(dtype=2))])
def test_rotary_refusals(code, change):
    refused(w4.w4a16_rotary, code, *{**ROTARY, **change}.values())


def test_workspace():
    f, r = w4.w4a16_kv4_tree_workspace_bytes, random.Random(3)
    assert f(0, 1, 1, 20, 8, 1, 128) == 0 and f(1, 4, 4, 20, 8, 1, 128, -1) == 0
    wide = 0
    for _ in range(20000):
        batch, new, D = int(2 ** r.uniform(0, 11)), int(2 ** r.uniform(0, 12)), r.choice([64, 128])
        kv, ratio = r.choice([1, 2, 5, 8, 32]), r.choice([1, 2, 4, 5, 8, 16])
        got = f(batch, r.randint(new, batch * new), new, int(2 ** r.uniform(0, 17)), kv * ratio, kv, D, r.choice([0, 0, 100, 5000]))
        assert got <= 4 * (512 + 1024 * 128 * (D + 2) + 512 * 8), (batch, new, kv, ratio)  # what a stream's own buffer is made to hold
        wide += got > 4 * (512 + 1024 * 16 * (D + 2))
    assert wide > 1000


def test_constants_match_the_header():
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "w4a16.h")).read()
    for name, value in (("HALVES", w4.ROTARY_HALVES), ("NEIGHBOURS", w4.ROTARY_NEIGHBOURS)):
        assert int(re.search(rf"#define W4A16_ROTARY_{name}\s+(\d+)", text).group(1)) == value
