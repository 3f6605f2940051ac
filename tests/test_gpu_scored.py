"""attn_scored, attn_tree and tree_accept on the GPU against the float64 oracle
on the cache's own bytes: every head dim, tier and rotation, head ratios, one
token to prompts, ragged and empty sequences, masks that leave rows empty,
unwritten positions (NaN bytes), split counts and merges, types, streams and
graphs.

Tolerance of a row: 2e-3 of its largest value (the library's bound: fp16
probabilities, the fp16 centroid table) plus the output type's rounding, half a
step. lse: 2e-3 + 1e-5 |lse|.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import compressed_kv_attention_gb300 as ckv  # noqa: E402
from compressed_kv_attention_gb300 import inputs  # noqa: E402
from oracle import scored as S  # noqa: E402
from tests import helpers as H  # noqa: E402
from tests.scored_cases import Cache, random_tree  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]
DEV = "cuda"
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def check(out, lse, o_ref, l_ref, what):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(l), empty), f"{what}: empty rows differ"
    assert np.all(o[empty] == 0.0) and np.all(np.isfinite(o)), what
    err, top = np.abs(o - o_ref).max(-1), np.abs(o_ref).max(-1)
    bad = err > (H.ATOL_REL + HALF_STEP[out.dtype]) * top
    assert not bad.any(), f"{what}: worst row {np.max(err / np.maximum(top, 1e-30)):.3e}, {int(bad.sum())} rows"
    f = ~empty
    assert np.all(np.abs(l[f] - l_ref[f]) <= H.LSE_ATOL + H.LSE_RTOL * np.abs(l_ref[f])), f"{what}: lse"


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32, device=DEV)


def run(c, lens, q, *, masks=None, cap=0.0, window=0, alibi=False, prefix=None, doc=None, n_of=None, n_split=0,
        out_type=torch.float32, stream=None, max_seq_len=None):
    B, n_q, Hq, D = q.shape
    out = torch.full(q.shape, float("nan"), dtype=out_type, device=DEV)
    lse = torch.full(q.shape[:3], float("nan"), device=DEV)
    m = max_seq_len if max_seq_len is not None else max(max(lens), 1)
    size = ckv.attn_tree_workspace if masks is not None else ckv.attn_scored_workspace
    ws = torch.zeros(size(c.packed, m, n_q, Hq, n_split), dtype=torch.uint8, device=DEV)
    kw = dict(softcap=cap, window=window, slopes=slopes_of(Hq) if alibi else None,
              q_len=None if n_of is None else ints(n_of), n_split=n_split, stream=stream)
    if masks is not None:
        mt = torch.from_numpy(np.ascontiguousarray(masks).view(np.int64)).to(DEV)
        ckv.attn_tree(c.packed, ints(lens), m, mt, q, 1 / math.sqrt(D), out, lse, ws, **kw)
    else:
        ckv.attn_scored(c.packed, ints(lens), m, q, 1 / math.sqrt(D), out, lse, ws,
                        prefix_len=None if prefix is None else ints(prefix),
                        doc_start=None if doc is None else ints(doc), **kw)
    return out, lse, ws


def reference(c, lens, q, *, masks=None, cap=0.0, window=0, alibi=False, prefix=None, doc=None, n_of=None, **_):
    B, n_q, Hq, D = q.shape
    qn = q.double().cpu().numpy()
    o, l = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    sl = slopes_of(Hq).double().cpu().numpy() if alibi else None
    for b in range(B):
        T, n = lens[b], n_q if n_of is None else n_of[b]
        if masks is not None:
            rows = S.tree_rows(T, masks[b, :n], window)
        else:
            rows = S.causal_rows(T, n, window, 0 if prefix is None else min(prefix[b], T),
                                 None if doc is None else doc[b][:n])
        o[b, :n], l[b, :n] = S.scored_attention(qn[b, :n], c.k[b][:, :T], c.v[b][:, :T], *rows, 1 / math.sqrt(D), cap, sl)
    return o, l


def queries(B, n_q, Hq, D, seed, dtype=torch.float16):
    outl = inputs.outlier_channels(D, max(1, D // 100), seed)
    return inputs.normal_tensor((B, n_q, Hq, D), seed, "q", outl, dtype=str(dtype)[6:], torch_out=True).to(DEV)


def compare(c, lens, q, what, **kw):
    out, lse, ws = run(c, lens, q, **kw)
    check(out, lse, *reference(c, lens, q, **kw), what)
    assert ckv.read_device_flag(ws) == 0
    return out, lse


TIERS = [(64, 2, False), (64, 3, False), (64, 4, False), (128, 3, False), (128, 2, True), (128, 4, False),
         (256, 3, False), (256, 4, True), (256, 2, False), (512, 3, False), (512, 4, False), (512, 2, True),
         (512, 3, True), (512, 4, True), (128, 3, True), (256, 3, True)]


@pytest.mark.parametrize("D,bits,rot", TIERS)
def test_every_tier_with_every_modification(D, bits, rot):
    lens = [407, 33, 130]
    c = Cache(D, 2, lens, 448, bits, rot, seed=D + bits)
    for n_q, Hq, kw in [(1, 2, dict(cap=5.0)), (3, 6, dict(alibi=True, n_split=3)),
                        (7, 16, dict(cap=20.0, window=50, alibi=True)),
                        (30, 8, dict(doc=[[max(0, (T - 30 + i) // 19 * 19) for i in range(30)] for T in lens])),
                        (33, 4, dict(prefix=[390, 20, 0], cap=30.0, n_split=2))]:
        compare(c, lens, queries(3, n_q, Hq, D, n_q), f"scored {D} {bits} {rot} {n_q} {kw}", **kw)
    masks = np.stack([np.pad(random_tree(n, np.random.default_rng(n)), (0, 21 - n)) for n in (21, 5, 13)])
    for Hq, kw in [(2, {}), (16, dict(window=6, alibi=True, cap=15.0, n_split=4))]:
        compare(c, lens, queries(3, 21, Hq, D, 5), f"tree {D} {bits} {rot} {kw}", masks=masks, n_of=[21, 5, 13], **kw)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1023])
@pytest.mark.parametrize("D", [64, 512])
def test_lengths_around_tiles(T, D):
    c = Cache(D, 1, [T], 1040, seed=T)
    for n_q in sorted({1, min(T, 5), min(T, 40)}):
        for kw in (dict(cap=10.0, alibi=True), dict(window=max(1, T // 3)), dict(prefix=[T])):
            compare(c, [T], queries(1, n_q, 8, D, T), f"{T} {n_q} {kw}", **kw)
    n = min(T, 17)
    masks = random_tree(n, np.random.default_rng(T))[None]
    compare(c, [T], queries(1, n, 8, D, T), f"tree {T}", masks=masks, window=max(1, T // 2))


@pytest.mark.parametrize("n_split", [0, 1, 2, 5, 33, 300, 1024])
def test_split_counts_and_both_merges(n_split):
    D, lens = 128, [700, 0, 41]
    c = Cache(D, 2, [max(1, t) for t in lens], 704)
    q = queries(3, 5, 12, D, 4)
    kw = dict(cap=12.0, alibi=True, n_split=n_split)
    want = compare(c, lens, q, f"split {n_split}", **kw)
    ckv.set_concurrent_kernels(True)
    try:
        compare(c, lens, q, f"split {n_split} tree merge", **kw)
    finally:
        ckv.set_concurrent_kernels(False)
    again = run(c, lens, q, **kw)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])  # no order depends on timing


@pytest.mark.parametrize("n_split", [0, 1, 2, 7, 11, 40, 200])
@pytest.mark.parametrize("D,rot", [(64, False), (128, True), (512, False), (512, True)])
def test_tiles_at_every_split_count(D, rot, n_split):
    """More than 32 query rows per kv head (the tiles), shares with and without keys, both merges of the partials."""
    lens, n_of = [700, 0, 41, 320], [20, 5, 20, 3]
    c = Cache(D, 2, [max(1, t) for t in lens], 704, rot=rot)
    q = queries(4, 20, 12, D, 4)
    kw = dict(cap=12.0, alibi=D == 128, n_split=n_split, n_of=n_of, window=300)
    want = compare(c, lens, q, f"tiles {D} {n_split}", **kw)
    again = run(c, lens, q, **kw)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    for out_type in (torch.float16, torch.bfloat16):
        compare(c, lens, q, f"tiles {D} {n_split} {out_type}", out_type=out_type, **kw)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_prompts_of_several_tiles(D):
    """A whole prompt and the last chunk of one: query tiles that end inside a document, a prefix, an odd last tile."""
    T = 333
    c = Cache(D, 1, [T, 290], 336, seed=D)
    starts = np.array([0, 37, 38, 129, 250])
    for n_q, Hq in ((290, 8), (131, 3)):
        q = queries(2, n_q, Hq, D, n_q, torch.bfloat16)
        doc = [starts[np.searchsorted(starts, np.arange(t - n_q, t), side="right") - 1] for t in (T, 290)]
        for kw in (dict(doc=doc), dict(prefix=[200, 290], cap=30.0), dict(window=65, alibi=True, doc=doc)):
            compare(c, [T, 290], q, f"prompt {D} {n_q} {list(kw)}", out_type=torch.bfloat16, **kw)


def test_probabilities_after_the_largest_logit_moves():
    """Keys whose logits climb along the sequence: the running maximum and the accumulated rows are rescaled often."""
    for D, n_q in ((128, 1), (128, 24), (512, 12)):
        c = Cache(D, 1, [640], 640, seed=9)
        q = queries(1, n_q, 4, D, 3)
        c.k[0] *= np.linspace(0.1, 6.0, 640)[None, :, None]
        k = torch.from_numpy(c.k[0].transpose(1, 0, 2)[None].astype(np.float16)).to(DEV)
        v = inputs.normal_tensor((1, 640, 1, D), 9, "v", np.zeros(0, np.int64))
        ckv.kv_pack(c.packed, 0, k.contiguous(), torch.from_numpy(v).to(DEV))
        c.read()
        compare(c, [640], q, f"climbing {D} {n_q}")
        compare(c, [640], q, f"climbing {D} {n_q}", alibi=True, n_split=3)


@pytest.mark.parametrize("rot", [False, True])
def test_unwritten_positions_and_left_padding(rot):
    """Positions before the padding's end and after the length are NaN bytes and must not be seen."""
    D, lens, start = 128, [210, 77, 19], [100, 13, 18]
    c = Cache(D, 1, lens, 256, 3, rot, start=start, seed=3)
    for n_q in (1, 6, 40):
        doc = [[start[b]] * n_q for b in range(3)]
        kw = dict(doc=doc, cap=9.0, alibi=True)
        out, lse = compare(c, lens, queries(3, n_q, 4, D, 9), f"padded {n_q}", **kw)
        if n_q == 40:  # rows inside the padding see nothing
            assert torch.isneginf(lse[2, :38]).all() and not torch.isneginf(lse[2, 39]).any()


@pytest.mark.parametrize("rot", [False, True])
def test_gaps_no_row_sees_may_hold_any_bytes(rot):
    """Two documents' windows leave a gap that no row sees: its bytes are NaN, inside the rows' common span."""
    D, T = 256, 200
    c = Cache(D, 1, [T], 208, 3, rot, seed=6)
    rec = c.packed.data.view(1, 13, -1)
    rec[0, 4] = 0xFF  # positions 64 .. 79
    doc = [[80 if i >= 128 else 0 for i in range(T)]]
    q = queries(1, T, 2, D, 2)
    out, lse, ws = run(c, [T], q, doc=doc, window=50)
    o, l = reference(c, [T], q, doc=doc, window=50)
    keep = np.array([not (p - 49 <= 79 and p >= 64 and p < 128) for p in range(T)])  # rows 64 .. 127 read the gap
    check(out[:, keep], lse[:, keep], o[:, keep], l[:, keep], "gap")


def test_empty_rows():
    D = 128
    c = Cache(D, 2, [60, 60, 60, 60], 64)
    q = queries(4, 6, 4, D, 1)
    lens, n_of = [0, 60, 3, 60], [6, 0, 6, 2]  # an empty sequence, no queries, more queries than positions, padded rows
    out, lse = compare(c, lens, q, "empty", n_of=n_of, cap=4.0)
    assert torch.isneginf(lse[0]).all() and torch.isneginf(lse[1]).all() and torch.isneginf(lse[2, :3]).all()
    compare(c, [60] * 4, q, "documents after every query", doc=[[60] * 6, [1000] * 6, [59] * 6, [-5] * 6])
    compare(c, [60] * 4, q, "prefixes", prefix=[-3, 0, 59, 10 ** 9], doc=[[58] * 6, [10] * 6, [57] * 6, [0] * 6])
    # A tree over an empty cache: nodes without bits see nothing.
    masks = np.zeros((4, 6), np.uint64)
    masks[1] = [1, 3, 0, 9, 0, 32]
    out, lse = compare(c, [6, 6, 60, 6], q, "tree", masks=masks, window=3)
    assert torch.isneginf(lse[0]).all() and torch.isneginf(lse[1, 2]).all() and not torch.isneginf(lse[1, 5]).any()


def test_tree_windows_count_depths():
    """A drafted ancestor further along the cache than the window is seen when its depth is near enough."""
    D, T, n = 64, 90, 64
    c = Cache(D, 1, [T], 96)
    rng = np.random.default_rng(0)
    q = queries(1, n, 8, D, 3)
    for width in (1, 4, 30):
        masks = random_tree(n, rng, width)[None]
        for window in (1, 2, 5, 30, 63, 64, 70):
            compare(c, [T], q, f"{width} {window}", masks=masks, window=window, alibi=True)
    compare(c, [64], q, "no committed keys", masks=random_tree(n, rng, 5)[None], window=4)
    full = np.full((1, n), 0xFFFFFFFFFFFFFFFF, np.uint64)  # not a tree: every node sees every node
    compare(c, [T], q, "all bits", masks=full)
    compare(c, [T], q[:, :9].contiguous(), "bits past the nodes", masks=np.full((1, 9), 0x1FF, np.uint64))


@pytest.mark.parametrize("out_type", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("q_type", [torch.float16, torch.bfloat16])
def test_types(q_type, out_type):
    for D in (128, 512):
        c = Cache(D, 2, [300, 11], 304)
        for n_q, n_split in ((1, 1), (1, 4), (9, 0)):
            compare(c, [300, 11], queries(2, n_q, 8, D, 8, q_type), f"{q_type} {out_type}", out_type=out_type,
                    n_split=n_split, cap=25.0)


@pytest.mark.parametrize("Hkv,Hq", [(1, 1), (3, 3), (2, 14), (1, 40), (8, 8), (1, 128), (1, 136)])
def test_head_ratios(Hkv, Hq):
    c = Cache(64, Hkv, [129, 50], 144)
    for n_q in (1, 2, 11):
        compare(c, [129, 50], queries(2, n_q, Hq, 64, 2), f"{Hkv} {Hq} {n_q}", cap=8.0, window=40)


def test_out_of_range_lengths_are_flagged_and_empty():
    c = Cache(128, 1, [40, 40], 48)
    q = queries(2, 3, 2, 128, 0)
    for lens, n_of, m in [([49, 40], None, 64), ([-1, 40], None, 48), ([41, 40], None, 40), ([40, 40], [4, 3], 48),
                          ([40, 40], [-1, 3], 48)]:
        out, lse, ws = run(c, lens, q, n_of=n_of, max_seq_len=m)
        assert ckv.read_device_flag(ws) == 2
        assert torch.isneginf(lse[0]).all() and (out[0] == 0).all() and torch.isfinite(lse[1]).all()
    out, lse, ws = run(c, [2, 40], q, masks=np.full((2, 3), 7, np.uint64))  # more nodes than positions
    assert ckv.read_device_flag(ws) == 2 and torch.isneginf(lse[0]).all() and torch.isfinite(lse[1]).all()


def test_wrong_tensors_are_refused():
    c = Cache(128, 1, [40], 48)
    q = queries(1, 3, 2, 128, 0)
    out, lse, ws = run(c, [40], q)
    sl = ints([40])
    bad = [dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(out=out[:, :2]), dict(lse=lse.half()),
           dict(seq_len=sl.long()), dict(slopes=slopes_of(4)), dict(doc_start=ints([[0, 0]])),
           dict(prefix_len=ints([1, 2])), dict(q_len=ints([[3]]))]
    for window in (-1, 2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            ckv.attn_scored(c.packed, sl, 40, q, 0.1, out, lse, ws, window=window)
    with pytest.raises(ValueError):
        ckv.attn_scored(c.packed, sl.cpu(), 40, q, 0.1, out, lse, ws)
    with pytest.raises(ValueError):
        ckv.tree_accept(c.packed, sl, 3, ints([[0, 1]]), ints([2]).cpu(), ints([0]))
    for kw in bad:
        a = dict(seq_len=sl, q=q, out=out, lse=lse, slopes=None, doc_start=None, prefix_len=None, q_len=None)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            ckv.attn_scored(c.packed, a["seq_len"], 40, a["q"], 0.1, a["out"], a["lse"], ws, slopes=a["slopes"],
                            doc_start=a["doc_start"], prefix_len=a["prefix_len"], q_len=a["q_len"])


def test_large_caps_slopes_and_logits():
    """Caps near zero and far above the logits, steep slopes, logits in the hundreds."""
    c = Cache(128, 1, [500], 512)
    q = queries(1, 4, 4, 128, 7) * 8
    for kw in (dict(cap=0.01), dict(cap=1e4), dict(cap=200.0, alibi=True), dict(alibi=True)):
        compare(c, [500], q, str(kw), **kw)


# ----------------------------------------------------------------- accept --

def spoil(c, at, k=None, v=None):
    """Position `at` of every sequence packed again with one value of K or V (dim 5) replaced."""
    x = {}
    for name, bad in (("k", k), ("v", v)):
        row = inputs.normal_tensor((len(c.lens), 1, c.Hkv, c.D), at, name, np.zeros(0, np.int64))
        if bad is not None:
            row[..., 5] = bad
        x[name] = torch.from_numpy(row).to(DEV)
    ckv.kv_pack(c.packed, at, x["k"], x["v"])
    c.read()


@pytest.mark.parametrize("n_q,Hq", [(6, 4), (5, 16), (40, 4)])
@pytest.mark.parametrize("D,bits,rot", [(128, 3, True), (256, 2, True), (512, 4, True), (512, 3, False), (64, 3, False)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(D, bits, rot, n_q, Hq):
    T = 200
    cases = [(T - 3, {}), (100, dict(doc=[[0 if i % 2 else 101 for i in range(n_q)]])), (T - 32, dict(window=30)),
             (T - 2, dict(prefix=[T - 1], cap=20.0, alibi=True)), (T - n_q + 2, "tree")]
    for at, kw in cases:
        for bad in (dict(v=math.inf), dict(v=math.nan), dict(k=math.inf)):
            c = Cache(D, 2, [T], 208, bits, rot, seed=at)
            spoil(c, at, **bad)
            q = queries(1, n_q, Hq, D, at)
            if kw == "tree":
                masks = random_tree(n_q, np.random.default_rng(n_q), width=4)[None]
                args, see = dict(masks=masks), S.tree_rows(T, masks[0])[2]
            else:
                args = kw
                see = S.causal_rows(T, n_q, kw.get("window", 0), kw.get("prefix", [0])[0], kw.get("doc", [None])[0])[2]
            clean = ~see[:, at]
            for n_split in (0, 1, 3):
                out, lse, ws = run(c, [T], q, n_split=n_split, **args)
                with np.errstate(invalid="ignore", over="ignore"):
                    o_ref, l_ref = reference(c, [T], q, **args)
                what = f"{D} {bits} {rot} {at} {args} {bad} {n_split}"
                check(out[:, clean], lse[:, clean], o_ref[:, clean], l_ref[:, clean], what)
                if "v" in bad:  # the sums do not read V
                    seen = ~torch.isfinite(out[:, ~clean]).all(-1)
                    assert seen.all(), what
                    assert np.allclose(lse.cpu().numpy(), l_ref, rtol=H.LSE_RTOL, atol=H.LSE_ATOL), what
                assert ckv.read_device_flag(ws) == 0


@pytest.mark.parametrize("n_split", [0, 1, 5, 40])
@pytest.mark.parametrize("D,rot,n_q", [(128, True, 5), (512, False, 1), (64, False, 30), (512, True, 40)])
def test_nan_queries_give_nan_rows(D, rot, n_q, n_split):
    T = 700
    c = Cache(D, 2, [T, 0], 704, 3, rot)
    q = queries(2, n_q, 8, D, 3)
    want = run(c, [T, 0], q, cap=25.0, n_split=n_split)[:2]
    q[0, n_q // 2, 3, 7] = math.nan
    q[1, 0, 0, 0] = math.nan  # an empty row: stays empty
    def same():
        out, lse, ws = run(c, [T, 0], q, cap=25.0, n_split=n_split)
        assert torch.isnan(out[0, n_q // 2, 3]).all() and torch.isnan(lse[0, n_q // 2, 3])
        out[0, n_q // 2, 3], lse[0, n_q // 2, 3] = want[0][0, n_q // 2, 3], want[1][0, n_q // 2, 3]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert ckv.read_device_flag(ws) == 0
    same()
    ckv.set_concurrent_kernels(True)
    try:
        want = run(c, [T, 0], torch.where(torch.isnan(q), torch.zeros_like(q), q), cap=25.0, n_split=n_split)[:2]
        same()
    finally:
        ckv.set_concurrent_kernels(False)


def accept(c, lens, n_q, path, count, n_of=None, stream=None):
    new, flag = ints([-7] * len(lens)), ints([0])
    ckv.tree_accept(c.packed, ints(lens), n_q, ints(path), ints(count), new, q_len=None if n_of is None else ints(n_of),
                    flag=flag, stream=stream)
    torch.cuda.synchronize()
    return new.tolist(), int(flag)


@pytest.mark.parametrize("D,bits,rot", TIERS)
def test_accept_moves_every_bit(D, bits, rot):
    lens, n_q = [200, 64, 77, 33], 64
    n_of = [64, 64, 21, 1]
    c = Cache(D, 2, lens, 208, bits, rot, seed=bits)
    rng = np.random.default_rng(D)
    for trial in range(4):
        before = [[c.fields(b, h, 208) for h in range(2)] for b in range(4)]
        m = [1, 5, 40, 64][trial]
        path = np.full((4, m), -1)
        count = []
        for b, n in enumerate(n_of):
            L = int(rng.integers(0, m + 1))
            p = rng.integers(0, n, L)  # any order, repeats, sources that are targets
            path[b, :L] = np.sort(p) if trial % 2 else p
            count.append(L)
        L1 = [t - n + k for t, n, k in zip(lens, n_of, count)]
        if max(L1[b] for b in range(4)) > 208:
            continue
        new, flag = accept(c, lens, n_q, path, count, n_of)
        assert new == L1 and flag == 0
        for b in range(4):
            where = np.arange(208)
            base = lens[b] - n_of[b]
            where[base:base + count[b]] = base + path[b, :count[b]]
            for h in range(2):
                for was, now in zip(before[b][h], c.fields(b, h, 208)):
                    assert np.array_equal(was[where], now), (trial, b, h)


def test_accept_leaves_bad_sequences_alone():
    lens, n_q = [40, 40, 40, 40, 40], 8
    c = Cache(128, 2, lens, 48)
    before = c.records().copy()
    path = np.array([[0, 8], [0, -1], [3, 2], [0, 1], [5, 1]])
    new, flag = accept(c, [40, 40, 3, 40, 49], n_q, path, [2, 2, 2, 3, 1])
    assert new == [40, 40, 3, 40, 49] and flag == 2
    assert np.array_equal(before, c.records())
    new, flag = accept(c, lens, n_q, path, [1, 0, 0, 2, 0], [8, 8, 9, 8, 8])
    assert new == [33, 32, 40, 34, 32] and flag == 2
    assert np.array_equal(before, c.records())


# ------------------------------------------------------------- as used --

def _step(c, lens, q, masks, path, count, q1, bufs):
    """Verify a tree, accept its path, attend the next token over the new lengths."""
    out, lse, ws, new, out1, lse1, ws1 = bufs
    D, n = q.shape[3], q.shape[1]
    ckv.attn_tree(c.packed, lens, 256, masks, q, 1 / math.sqrt(D), out, lse, ws, softcap=20.0, window=100)
    ckv.tree_accept(c.packed, lens, n, path, count, new)
    ckv.attn_scored(c.packed, new, 256, q1, 1 / math.sqrt(D), out1, lse1, ws1, softcap=20.0, window=100)


def test_tree_accept_and_next_token_together_also_captured():
    D, lens, n = 128, [250, 90], 12
    rng = np.random.default_rng(4)
    masks = np.stack([random_tree(n, rng) for _ in lens])
    q, q1 = queries(2, n, 8, D, 1), queries(2, 1, 8, D, 2)
    path, count = np.array([[0, 2, 5, 11], [0, 1, 7, -1]]), [4, 3]
    results = []
    for captured in (False, True):
        c = Cache(D, 2, lens, 256, seed=8)
        bufs = (torch.empty_like(q), torch.empty(2, n, 8, device=DEV),
                torch.zeros(ckv.attn_tree_workspace(c.packed, 256, n, 8), dtype=torch.uint8, device=DEV),
                ints([0, 0]), torch.empty_like(q1), torch.empty(2, 1, 8, device=DEV),
                torch.zeros(ckv.attn_scored_workspace(c.packed, 256, 1, 8), dtype=torch.uint8, device=DEV))
        t = (ints(lens), q, torch.from_numpy(masks.view(np.int64)).to(DEV), ints(path), ints(count), q1)
        saved = c.packed.data.clone()
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                _step(c, *t, bufs)
            torch.cuda.current_stream().wait_stream(side)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                _step(c, *t, bufs)
            for _ in range(3):
                c.packed.data.copy_(saved)
                g.replay()
        else:
            _step(c, *t, bufs)
        torch.cuda.synchronize()
        results.append([x.clone() for x in (bufs[0], bufs[1], bufs[3], bufs[4], bufs[5], c.packed.data)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    out, lse, new, out1, lse1, _ = results[0]
    assert new.tolist() == [242, 81]
    c = Cache(D, 2, lens, 256, seed=8)
    kw = dict(masks=masks, cap=20.0, window=100)
    check(out, lse, *reference(c, lens, q, **kw), "tree")
    for b in range(2):
        w = S.accepted_positions(lens[b], n, path[b, :count[b]])
        c.k[b], c.v[b] = c.k[b][:, w], c.v[b][:, w]
    check(out1, lse1, *reference(c, [242, 81], q1, cap=20.0, window=100), "next token")


def test_two_streams_with_their_own_workspaces():
    c = Cache(256, 2, [900], 912)
    qs = [queries(1, n, 8, 256, n) for n in (1, 17)]
    want = [run(c, [900], q, cap=30.0)[:2] for q in qs]
    torch.cuda.synchronize()
    ckv.set_concurrent_kernels(True)
    try:
        streams = [torch.cuda.Stream() for _ in qs]
        got = []
        for s, q in zip(streams, qs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run(c, [900], q, cap=30.0)[:2])
        torch.cuda.synchronize()
    finally:
        ckv.set_concurrent_kernels(False)
    for q, (o, l), (o2, l2) in zip(qs, want, got):
        check(o2, l2, *reference(c, [900], q, cap=30.0), "stream")
