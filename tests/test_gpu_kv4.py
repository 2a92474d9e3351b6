"""The 4-bit KV cache on the GPU against its definition in 64 bits (needs a B200)."""

import numpy as np
import pytest
import torch

import synth
from synth import configs
from tests import _harness as H
from tests import _kv4 as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_megakernel_02_b200 import build

    build.build()


class Setup:
    """A cache filled with NaN bytes, a batch over it, and the numbers in numpy."""

    def __init__(self, d, kv_heads, lens, new, layers=1, pad_rows=0, seed=0, slack=0):
        from persistent_megakernel_02_b200 import Kv4Cache

        self.rng = np.random.default_rng(seed)
        self.d, self.kv_heads, self.lens, self.new = d, kv_heads, list(lens), list(new)
        self.table_np, pages = R.tables([max(v, 1) for v in lens], self.rng)
        self.table = torch.from_numpy(self.table_np).cuda()
        self.cache = Kv4Cache.empty(layers, pages, kv_heads, d, self.table)
        self.cache.pool.fill_(255)  # scales and minima of 0xFFFF are NaN
        self.cu_np = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.cu = torch.from_numpy(self.cu_np).cuda()
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.rows = int(self.cu_np[-1]) + pad_rows
        self.max_len = min(max(lens) + slack, R.PAGE * self.table_np.shape[1])
        self.batch = self.cache.batch(self.cu, self.kv_lens, self.rows, max(new), self.max_len)

    def full_batch(self):
        cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        t = torch.from_numpy(cu).cuda()
        return self.cache.batch(t, self.kv_lens, int(cu[-1]), max(self.lens), max(self.lens))

    def rand(self, rows, heads, dtype="fp32", spread=None):
        x = self.rng.standard_normal((rows, heads, self.d))
        if spread is not None:
            x = x * spread
        return torch.from_numpy(x).to(R.DTYPES[dtype]).cuda()

    def fill(self, layer=0, keys=1.0):
        """Every position of every sequence; returns K, V (float64) per sequence."""
        b = self.full_batch()
        gain = np.ones(self.d)
        gain[3] = 5.0
        k, v = self.rand(b.n_rows, self.kv_heads, spread=keys * gain), self.rand(b.n_rows, self.kv_heads)
        if b.n_rows:
            self.cache.append(layer, k, v, b)
        out, at = [], 0
        for n in self.lens:
            out.append(tuple(R.quantised(x[at:at + n].double().cpu().numpy()) for x in (k, v)))
            at += n
        return out

    def pool(self):
        return self.cache.pool.cpu().numpy()

    def pages(self, i):
        return self.table_np[i, : -(-self.lens[i] // R.PAGE)]


def reference(s, kv, q, i, scale):
    """(out, reach) of sequence i (see _kv4.attention), in 64 bits on the GPU a kv head at a time."""
    n_len, n = s.lens[i], s.new[i]
    a, b = s.cu_np[i], s.cu_np[i + 1]
    k, v = (torch.from_numpy(x).cuda() for x in kv[i])
    heads, rep = q.shape[1], q.shape[1] // s.kv_heads
    out = torch.zeros((n, heads, s.d), dtype=torch.float64, device="cuda")
    reach = torch.zeros((n, heads), dtype=torch.float64, device="cuda")
    see = torch.arange(n_len, device="cuda")[None, :] <= torch.arange(n_len - n, n_len, device="cuda")[:, None]
    some = see.any(-1)
    for h in range(heads if n_len and n else 0):
        x, kk, vv = q[a:b, h].double(), k[:, h // rep], v[:, h // rep]
        sc = (x @ kk.T * scale).masked_fill(~see, -np.inf)
        out[some, h] = torch.softmax(sc[some], -1) @ vv
        reach[:, h] = (x.abs() @ kk.abs().T * abs(scale)).masked_fill(~see, 0).amax(-1)
    return out.cpu().numpy(), reach.cpu().numpy()


def check_attention(s, kv, q, out, dtype, scale=None):
    scale = R.default_scale(s.d) if scale is None else scale
    on = out.double().cpu().numpy()
    for i, (n_len, n) in enumerate(zip(s.lens, s.new)):
        a, b = s.cu_np[i], s.cu_np[i + 1]
        if a == b:
            continue
        want, reach = reference(s, kv, q, i, scale)
        v_max = np.abs(kv[i][1]).max() if n_len else 0.0
        err = np.abs(on[a:b] - want)
        tol = R.tolerance(want, reach, v_max, dtype)
        assert np.isfinite(on[a:b]).all(), f"sequence {i}"
        assert (err <= tol).all(), f"sequence {i}: error {err.max():.3e}, worst ratio {(err / tol).max():.2f}"


# ---- writing and reading ------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,kv_heads", [(64, 8), (128, 1), (128, 3)])
@pytest.mark.parametrize("lens,new", [
    ([1], [1]), ([16], [16]), ([17, 64, 65], [17, 64, 65]), ([130, 5, 77, 1], [1, 5, 30, 0]),
    ([63, 128, 200], [62, 100, 137]),
])
def test_append_and_read_match_the_definition(d, kv_heads, lens, new, dtype):
    s = Setup(d, kv_heads, lens, new, pad_rows=3)
    k, v = s.rand(s.rows, kv_heads, dtype, spread=3.0), s.rand(s.rows, kv_heads, dtype)
    before = s.pool()
    s.cache.append(0, k, v, s.batch)
    ko, vo = (torch.full_like(k, -7.0) for _ in range(2))
    s.cache.read(0, ko, vo, s.batch)
    s.cache.check()
    after = s.pool()
    used = np.zeros(after.shape[1], bool)
    for i in range(len(lens)):
        a, b = s.cu_np[i], s.cu_np[i + 1]
        start = lens[i] - new[i]
        kk, vv = R.unpack(after, 0, s.pages(i), lens[i])
        assert np.isnan(kk[:start]).all() and np.isnan(vv[:start]).all()  # earlier positions as they were
        for x, stored, back in ((k, kk, ko), (v, vv, vo)):
            want = R.quantised(x[a:b].double().cpu().numpy())
            assert np.array_equal(stored[start:], want)
            assert torch.equal(back[a:b].cpu(), torch.from_numpy(want).to(torch.float32).to(R.DTYPES[dtype]))
        used[s.pages(i)[start // R.PAGE:]] = True
    assert np.array_equal(after[:, ~used], before[:, ~used])  # no other page is touched
    for t in (ko, vo):
        assert (t[s.cu_np[-1]:] == -7.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_append_decides_ties_and_edges_exactly(dtype):
    """Rows on and next to the borders between codes, constant rows, tiny and huge ranges."""
    s = Setup(64, 2, [64], [64])
    x = np.zeros((64, 2, 64))
    grid = np.arange(64)
    x[0, 0] = grid % 31 / 2                       # every border of a 0..15 grid, exactly half way
    x[1, 0] = -100 + grid % 31 / 2                # the same with an offset
    x[2, 0] = 3.25                                # constant
    x[3, 0] = 0.0
    x[4, 0] = grid * 2.0**-24                     # steps below fp16's smallest normal
    x[5, 0] = (grid - 31) * 1000.0
    x[6, 0] = np.where(grid % 2, 32768.0, -32768.0)
    x[7, 0] = grid % 31 / 2 + 1e-3                # next to the borders
    x[8, 0] = 1.0 + grid * 2.0**-7
    x[9, 0] = -(2.0 ** -(grid % 20))
    x[10:, :] = s.rng.standard_normal((54, 2, 64)) * 2.0 ** s.rng.integers(-12, 12, (54, 2, 1))
    x[11:20] = np.round(x[11:20] * 8) / 8         # coarse values make exact ties common
    k = torch.from_numpy(x).to(R.DTYPES[dtype]).cuda()
    v = k.flip(0).contiguous()
    s.cache.append(0, k, v, s.batch)
    got = R.unpack(s.pool(), 0, s.pages(0), 64)
    for t, g in zip((k, v), got):
        assert np.array_equal(g, R.quantised(t.double().cpu().numpy()))


def test_append_marks_groups_it_cannot_hold():
    s = Setup(64, 1, [16], [16])
    k, v = s.rand(16, 1), s.rand(16, 1)
    k[0, 0, 5], k[1, 0, 40], v[2, 0, 0], v[3, 0, 63] = float("nan"), float("inf"), -float("inf"), 40000.0
    s.cache.append(0, k, v, s.batch)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    s.cache.read(0, ko, vo, s.batch)
    s.cache.check()
    bad_k, bad_v = torch.zeros_like(k, dtype=torch.bool), torch.zeros_like(k, dtype=torch.bool)
    bad_k[0, 0, :32], bad_k[1, 0, 32:], bad_v[2, 0, :32], bad_v[3, 0, 32:] = True, True, True, True
    assert torch.equal(ko.isnan(), bad_k) and torch.equal(vo.isnan(), bad_v)


@pytest.mark.parametrize("layout", ["fused", "heads first", "one row for all"])
def test_rows_with_other_strides(layout):
    s = Setup(64, 4, [40], [40], layers=3)
    if layout == "fused":       # a fused projection's output: q, k and v side by side
        whole = s.rand(40, 16, "bf16")
        k, v = whole[:, 8:12], whole[:, 12:]
    elif layout == "heads first":
        whole = torch.stack([s.rand(40, 4, "bf16"), s.rand(40, 4, "bf16")])
        k, v = (whole[i].transpose(0, 1).contiguous().transpose(0, 1) for i in range(2))
    else:                       # broadcast inputs
        k, v = s.rand(1, 4, "bf16").expand(40, 4, 64), s.rand(40, 1, "bf16").expand(40, 4, 64)
    s.cache.append(1, k, v, s.batch)
    got = R.unpack(s.pool(), 1, s.pages(0), 40)
    for t, g in zip((k, v), got):
        assert np.array_equal(g, R.quantised(t.double().cpu().numpy()))
    assert (s.pool()[[0, 2]] == 255).all()
    out = torch.full((2, 4, 40, 64), -1.0, dtype=torch.bfloat16, device="cuda")  # heads first
    s.cache.read(1, out[0].transpose(0, 1), out[1].transpose(0, 1), s.batch)
    for o, g in zip(out, got):
        assert torch.equal(o.transpose(0, 1).cpu(), torch.from_numpy(g).float().bfloat16())


# ---- attention --------------------------------------------------------------------------

TOKENS = [([1], [1]), ([15], [1]), ([16, 17, 64, 65], [1] * 4), ([300, 1, 0, 1000], [1, 1, 0, 1]), ([5000], [1]),
          ([2100, 130], [1, 1])]
FEW = [([2], [2]), ([70, 16, 33], [3, 8, 1]), ([600], [16]), ([4000, 33], [5, 2]), ([40, 0, 9], [17, 0, 9])]
PROMPTS = [([33], [33]), ([200, 64, 1], [200, 64, 1]), ([513], [400]), ([700, 129], [100, 129])]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,kv_heads,rep", [(64, 2, 4), (128, 1, 8), (64, 3, 1), (128, 2, 2), (128, 2, 4)])
@pytest.mark.parametrize("lens,new", TOKENS + FEW + PROMPTS)
def test_attention_matches_the_definition(lens, new, d, kv_heads, rep, dtype):
    s = Setup(d, kv_heads, lens, new, pad_rows=2)
    kv = s.fill()
    q = s.rand(s.rows, kv_heads * rep, dtype)
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, q, out, s.batch)
    s.cache.check()
    check_attention(s, kv, q, out, dtype)
    assert (out[s.cu_np[-1]:] == -7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_rows_that_see_nothing_are_zero(dtype, n):
    """A span longer than its sequence: its first rows stand before position 0."""
    s = Setup(64, 2, [n - 1, 70], [n, 1])
    kv = s.fill()
    q = s.rand(s.rows, 8, dtype)
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, q, out, s.batch)
    s.cache.check()
    assert (out[0] == 0).all()
    check_attention(s, kv, q, out, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_attention_scales(dtype, new, scale):
    s = Setup(64, 2, [200], [new])
    kv = s.fill(keys=0.2)
    q = s.rand(s.rows, 4, dtype)
    out = torch.empty_like(q)
    s.cache.attend(0, q, out, s.batch, scale=scale)
    check_attention(s, kv, q, out, dtype, scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("k_size,q_size,v_size", [(2.0**-12, 2.0**10, 2.0**-9), (2.0**9, 2.0**-11, 2.0**9), (30.0, 1.0, 1.0)])
def test_attention_of_small_and_large_values(dtype, new, k_size, q_size, v_size):
    """Ranges far from 1, and scores far apart (one position takes all the weight)."""
    s = Setup(128, 1, [170], [new])
    b = s.full_batch()
    k, v = s.rand(170, 1, spread=k_size), s.rand(170, 1, spread=v_size)
    s.cache.append(0, k, v, b)
    kv = [tuple(R.quantised(x.double().cpu().numpy()) for x in (k, v))]
    q = s.rand(s.rows, 4, dtype, spread=q_size)
    out = torch.empty_like(q)
    s.cache.attend(0, q, out, s.batch)
    check_attention(s, kv, q, out, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new", [1, 70])
def test_nan_in_the_cache_reaches_only_the_rows_that_see_it(dtype, new):
    s = Setup(64, 2, [300], [new])
    s.fill()
    q = s.rand(s.rows, 8, dtype)
    clean = torch.empty_like(q)
    s.cache.attend(0, q, clean, s.batch)
    at = 300 - new // 2 - 1  # rows from this position on see it
    bad = s.cache.batch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                        torch.tensor([at + 1], dtype=torch.int32, device="cuda"), 1, 1, at + 1)
    one = torch.full((1, 2, 64), float("nan"), device="cuda")
    one[:, 1] = 1.0  # kv head 0 only
    s.cache.append(0, one, one, bad)
    out = torch.empty_like(q)
    s.cache.attend(0, q, out, s.batch)
    first = at - (300 - new)
    assert out[first:, :4].isnan().all()
    assert torch.equal(out[:first], clean[:first])
    assert not out[:, 4:].isnan().any()


# Enough rows for the tensor-memory kernel (16-bit types): whole and ragged blocks of 256 rows,
# rows that end inside a tile of 128, spans longer than their sequence, single tokens beside
# prompts, and few blocks over a long cache, which are split along it.
MANY = [([1000, 777, 130], [1000, 700, 129], 8, 4), ([513, 64, 1, 0, 300, 256, 128, 65], [513, 64, 1, 0, 299, 200, 128, 33], 8, 4),
        ([70, 400, 500, 380, 41, 450], [90, 380, 390, 1, 400, 2], 8, 4), ([6000], [600], 2, 4), ([5000, 3100], [333, 128], 1, 8),
        ([700] * 5, [430] * 5, 8, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,new,kv_heads,rep", MANY)
def test_attention_of_many_rows(lens, new, kv_heads, rep, d, dtype):
    s = Setup(d, kv_heads, lens, new, pad_rows=2)
    kv = s.fill()
    q = s.rand(s.rows, kv_heads * rep, dtype)
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, q, out, s.batch)
    s.cache.check()
    check_attention(s, kv, q, out, dtype)
    assert (out[s.cu_np[-1]:] == -7.0).all()
    again = torch.full_like(q, -7.0)
    s.cache.attend(0, q, again, s.batch)
    assert torch.equal(out, again)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_attention_of_many_rows_scales(scale):
    s = Setup(64, 8, [500] * 4, [400] * 4)
    kv = s.fill(keys=0.2)
    q = s.rand(s.rows, 32, "bf16")
    out = torch.empty_like(q)
    s.cache.attend(0, q, out, s.batch, scale=scale)
    check_attention(s, kv, q, out, "bf16", scale)


@pytest.mark.parametrize("k_size,q_size,v_size", [(2.0**-9, 2.0**7, 2.0**-7), (2.0**9, 2.0**-11, 2.0**9), (30.0, 1.0, 1.0)])
def test_attention_of_many_rows_small_and_large_values(k_size, q_size, v_size):
    s = Setup(128, 8, [420] * 3, [400] * 3)
    b = s.full_batch()
    k, v = s.rand(b.n_rows, 8, spread=k_size), s.rand(b.n_rows, 8, spread=v_size)
    s.cache.append(0, k, v, b)
    kv = [tuple(R.quantised(x[420 * i:420 * (i + 1)].double().cpu().numpy()) for x in (k, v)) for i in range(3)]
    q = s.rand(s.rows, 32, "fp16", spread=q_size)
    out = torch.empty_like(q)
    s.cache.attend(0, q, out, s.batch)
    check_attention(s, kv, q, out, "fp16")


@pytest.mark.parametrize("lens,new", [([500] * 4, [300] * 4), ([6000], [600])])
@pytest.mark.parametrize("where", ["keys", "values"])
def test_nan_in_a_prompt_reaches_only_the_rows_that_see_it(where, lens, new):
    """One position's K or V of kv head 0 is NaN in one group: later rows see it (all values for K,
    the group's for V), earlier ones and the other heads do not."""
    kvh = 8 if len(lens) > 1 else 2
    s = Setup(64, kvh, lens, new)
    s.fill()
    q = s.rand(s.rows, 4 * kvh, "bf16")
    clean, out = torch.empty_like(q), torch.empty_like(q)
    s.cache.attend(0, q, clean, s.batch)
    at = lens[0] - 77
    one = s.cache.batch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                        torch.tensor([at + 1], dtype=torch.int32, device="cuda"), 1, 1, at + 1)
    k, v = torch.empty((1, kvh, 64), device="cuda"), torch.empty((1, kvh, 64), device="cuda")
    s.cache.read(0, k, v, one)
    (k if where == "keys" else v)[0, 0, 40] = float("nan")
    s.cache.append(0, k, v, one)
    s.cache.attend(0, q, out, s.batch)
    first, end = at - (lens[0] - new[0]), new[0]
    bad = out[first:end, :4]
    assert bad.isnan().all() if where == "keys" else bad[..., 32:].isnan().all() and not bad[..., :32].isnan().any()
    assert torch.equal(out[:first], clean[:first]) and not out[:, 4:].isnan().any() and not out[end:].isnan().any()


def test_missing_pages_of_a_prompt_are_reported_and_masked():
    from persistent_megakernel_02_b200 import MkError

    s = Setup(64, 8, [500] * 4, [300] * 4)
    kv = s.fill()
    q = s.rand(s.rows, 32, "bf16")
    out = torch.empty_like(q)
    for page in (s.cache.n_pages, -1):
        s.table[1, 2] = page
        s.cache.attend(0, q, out, s.batch)
        with pytest.raises(MkError, match="DEVICE_FAULT"):
            s.cache.check()
        assert torch.isfinite(out).all()
    cu = s.cu_np
    for i in (0, 2, 3):  # the other sequences
        want, reach = reference(s, kv, q, i, R.default_scale(64))
        err = np.abs(out[cu[i]:cu[i + 1]].double().cpu().numpy() - want)
        assert (err <= R.tolerance(want, reach, np.abs(kv[i][1]).max(), "bf16")).all()
    k, v = (np.delete(x, slice(128, 192), 0) for x in kv[1])  # the rows behind it: as if it were not there
    x = q[cu[2] - 100:cu[2]]
    t = Setup(64, 8, [436], [100])
    want, reach = reference(t, [(k, v)], x, 0, R.default_scale(64))
    err = np.abs(out[cu[2] - 100:cu[2]].double().cpu().numpy() - want)
    assert (err <= R.tolerance(want, reach, np.abs(v).max(), "bf16")).all()


@pytest.mark.parametrize("d,kv_heads,new", [(64, 16, 400), (128, 16, 300), (64, 2, 400), (64, 8, 1), (64, 8, 40)])
def test_missing_pages_of_a_long_cache_are_left_out(d, kv_heads, new):
    """Pages missing here and there: each block is masked by its own page's flag."""
    from persistent_megakernel_02_b200 import MkError

    n_len, gone = 2500, (3, 10, 11, 18, 24, 31)  # all before the first query
    s = Setup(d, kv_heads, [n_len], [new])
    kv = s.fill()
    q = s.rand(s.rows, 2 * kv_heads, "bf16")
    out = torch.empty_like(q)
    for i, page in enumerate(gone):
        s.table[0, page] = s.cache.n_pages + i if i % 2 else -1 - i
    rest = np.concatenate([np.arange(64 * p, 64 * p + 64) for p in gone])
    kv = [tuple(np.delete(x, rest, 0) for x in kv[0])]
    t = Setup(d, kv_heads, [n_len - len(rest)], [new])  # the same as without them
    for _ in range(3):
        s.cache.attend(0, q, out, s.batch)
        with pytest.raises(MkError, match="DEVICE_FAULT"):
            s.cache.check()
        check_attention(t, kv, q, out, "bf16")


@pytest.mark.parametrize("new", [400, 1])
@pytest.mark.parametrize("page", [-1, -2, -3, -2**31, 2**31 - 1])
def test_every_page_id_outside_the_pool_is_reported(page, new):
    from persistent_megakernel_02_b200 import MkError

    s = Setup(64, 16, [1000], [new])
    s.fill()
    q = s.rand(s.rows, 32, "bf16")
    out = torch.empty_like(q)
    s.table[0, 3] = page
    s.cache.attend(0, q, out, s.batch)
    with pytest.raises(MkError, match="DEVICE_FAULT"):
        s.cache.check()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("kv_heads,lens,new", [(2, [90, 300], [40, 1]), (8, [500] * 4, [300] * 4)])
def test_attention_with_other_strides(kv_heads, lens, new):
    s = Setup(128, kv_heads, lens, new, layers=2)
    kv = s.fill(layer=1)
    whole = s.rand(s.rows, 4 * kv_heads + 4, "fp16")
    q = whole[:, 2:-2]
    out = torch.full((4 * kv_heads, s.rows, 128), -1.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    s.cache.attend(1, q, out, s.batch)
    check_attention(s, kv, q, out, "fp16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeated_calls_give_the_same_bits(dtype):
    s = Setup(64, 8, [3000, 700, 64], [1, 40, 2])
    s.fill()
    q = s.rand(s.rows, 32, dtype)
    a, b = torch.empty_like(q), torch.empty_like(q)
    s.cache.attend(0, q, a, s.batch)
    for _ in range(3):
        b.fill_(-1)
        s.cache.attend(0, q, b, s.batch)
        assert torch.equal(a, b)


def test_two_streams_and_a_given_workspace():
    s = Setup(64, 8, [6000, 2500], [1, 1])
    kv = s.fill()
    q = [s.rand(s.rows, 32, "bf16") for _ in range(2)]
    out = [torch.empty_like(x) for x in q]
    need = s.cache.workspace_bytes(s.batch, 32, torch.bfloat16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(need + 256, dtype=torch.uint8, device="cuda"), None]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, x, o, w in zip(streams, q, out, spaces):
            s.cache.attend(0, x, o, s.batch, workspace=w, stream=st)
    torch.cuda.synchronize()
    for x, o in zip(q, out):
        check_attention(s, kv, x, o, "bf16")


@pytest.mark.parametrize("new", [1, 50])
def test_a_captured_step_replays_as_the_sequence_grows(new):
    """append and attend in one CUDA graph; the lengths on the device grow between replays."""
    from persistent_megakernel_02_b200 import Kv4Cache

    d, kvh, heads, n0 = 64, 2, 8, 100
    total = n0 + 3 * new
    rng = np.random.default_rng(5)
    table = torch.from_numpy(R.tables([total + 64], rng)[0]).cuda()
    cache = Kv4Cache.empty(1, int(table.max()) + 1, kvh, d, table)
    cache.pool.fill_(255)
    rows = [torch.from_numpy(rng.standard_normal((total, h, d))).float().cuda() for h in (kvh, kvh, heads)]
    first = cache.batch(torch.tensor([0, n0], dtype=torch.int32, device="cuda"),
                        torch.tensor([n0], dtype=torch.int32, device="cuda"), n0, n0, n0)
    cache.append(0, rows[0][:n0], rows[1][:n0], first)
    k, v, q = (torch.zeros((new, h, d), device="cuda") for h in (kvh, kvh, heads))
    out = torch.empty_like(q)
    lens = torch.tensor([n0], dtype=torch.int32, device="cuda")
    batch = cache.batch(torch.tensor([0, new], dtype=torch.int32, device="cuda"), lens, new, new, total)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # the first call of a kernel outside the capture
        cache.attend(0, q, out, batch)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(0, k, v, batch)
        cache.attend(0, q, out, batch)
    kq, vq = (R.quantised(x.double().cpu().numpy()) for x in rows[:2])
    for step in range(3):
        a = n0 + step * new
        for dst, src in zip((k, v, q), rows):
            dst.copy_(src[a:a + new])
        lens.fill_(a + new)
        graph.replay()
        torch.cuda.synchronize()
        want, reach = R.attention(q.double().cpu().numpy(), kq[:a + new], vq[:a + new], a + new, R.default_scale(d))
        err = np.abs(out.double().cpu().numpy() - want)
        assert (err <= R.tolerance(want, reach, np.abs(vq).max(), "fp32")).all(), step
    cache.check()


@pytest.mark.parametrize("n_len,new,kv_heads", [(9000, 1, 2), (1500, 1, 16), (6000, 200, 2), (700, 300, 16)])
def test_a_captured_call_of_every_form_replays(n_len, new, kv_heads):
    """Splits joined by a second launch, by a cluster, a prompt split along the cache, a prompt not split: captured
    without a call before, replayed with other queries."""
    s = Setup(64, kv_heads, [n_len], [new])
    kv = s.fill()
    q = s.rand(s.rows, 4 * kv_heads, "bf16")
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attend(0, q, out, s.batch)
    for _ in range(2):
        q.copy_(s.rand(s.rows, 4 * kv_heads, "bf16"))
        out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(s, kv, q, out, "bf16")
    s.cache.check()


@pytest.mark.parametrize("lens,new,kv_heads", [([9000, 70], [1, 1], 2), ([1500], [1], 16), ([6000], [200], 2), ([700, 300], [300, 5], 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_output_may_be_the_queries(lens, new, kv_heads, dtype):
    s = Setup(64, kv_heads, lens, new)
    kv = s.fill()
    q = s.rand(s.rows, 4 * kv_heads, dtype)
    same = q.clone()
    s.cache.attend(0, same, same, s.batch)
    check_attention(s, kv, q, same, dtype)


def test_caches_of_other_shapes_share_a_batch():
    """Two models over the same sequences: the workspace is the called cache's."""
    from persistent_megakernel_02_b200 import Kv4Cache

    sets = [Setup(d, kvh, [9000], [1], seed=3) for d, kvh in ((64, 32), (64, 4), (128, 4))]
    shared = sets[0].batch
    needs = set()
    for s in sets + sets[::-1]:
        kv = s.fill()
        s.cache = Kv4Cache(s.cache.pool, s.table, s.d)
        q = s.rand(1, 32, "bf16")
        out = torch.empty_like(q)
        needs.add(s.cache.workspace_bytes(s.batch, 32, torch.bfloat16))
        s.cache.attend(0, q, out, shared)
        check_attention(s, kv, q, out, "bf16")
    assert len(needs) > 1


@pytest.mark.parametrize("new", [[2, 1], [300, 200]])
def test_rows_before_the_first_sequence_are_left_alone(new):
    """cu may start behind row 0: rows no sequence owns are neither read nor written."""
    s = Setup(64, 8, [400, 350], new)
    kv = s.fill()
    cu = s.cu + 3
    batch = s.cache.batch(cu, s.kv_lens, s.rows + 3, max(new), s.max_len)
    q = torch.cat([torch.full((3, 32, 64), float("nan"), dtype=torch.bfloat16, device="cuda"), s.rand(s.rows, 32, "bf16")])
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, q, out, batch)
    assert (out[:3] == -7.0).all()
    check_attention(s, kv, q[3:], out[3:], "bf16")
    k, v = (torch.full((s.rows + 3, 8, 64), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s.cache.read(0, k, v, batch)
    s.cache.check()
    assert (k[:3] == -7.0).all() and (v[:3] == -7.0).all()
    at = 3
    for (kk, vv), n in zip(kv, new):
        for t, x in ((k, kk), (v, vv)):
            assert torch.equal(t[at:at + n].cpu(), torch.from_numpy(x[len(x) - n:]).float().bfloat16())
        at += n


@pytest.mark.parametrize("where", ["current", "default by number", "side"])
def test_check_waits_for_its_stream(where):
    """The status is read behind the stream's work, also where that takes a while."""
    from persistent_megakernel_02_b200 import MkError

    s = Setup(64, 2, [40], [40])
    s.fill()
    q = s.rand(40, 8, "bf16")
    out = torch.empty_like(q)
    s.table[0, 0] = s.cache.n_pages
    work = torch.randn(8192, 8192, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    arg = {"current": None, "default by number": 0, "side": side}[where]
    with torch.cuda.stream(side if where == "side" else torch.cuda.default_stream()):
        for _ in range(30):  # over 20 ms
            work @ work
        s.cache.attend(0, q, out, s.batch, stream=arg)
    with pytest.raises(MkError, match="DEVICE_FAULT"):
        s.cache.check(stream=arg)
    s.cache.check(stream=arg)


# ---- what the device finds wrong ---------------------------------------------------------


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("what", ["length", "negative length", "span", "cu", "page"])
def test_numbers_out_of_bounds_are_reported_and_touch_nothing(what, new):
    """The host's own checks turn these into a status word; the other sequence is served."""
    from persistent_megakernel_02_b200 import MkError

    s = Setup(64, 2, [100, 90], [new, new])
    kv = s.fill()
    q = s.rand(s.rows, 8, "bf16")
    out = torch.full_like(q, -7.0)
    before = s.pool()
    if what == "length":
        s.kv_lens[0] = s.max_len + 1
    elif what == "negative length":
        s.kv_lens[0] = -1
    elif what == "span":
        s.batch = s.cache.batch(s.cu, s.kv_lens, s.rows, max(new - 1, 0), s.max_len)
    elif what == "cu":
        s.cu[0] = -1
    else:
        s.table[0, 0] = s.cache.n_pages
    k = s.rand(s.rows, 2, "bf16")
    s.cache.append(0, k, k, s.batch)
    if what != "page":
        with pytest.raises(MkError, match="DEVICE_FAULT"):
            s.cache.check()
        after = s.pool()
        assert np.array_equal(after[:, s.pages(0)], before[:, s.pages(0)])
    s.cache.attend(0, q, out, s.batch)
    with pytest.raises(MkError, match="DEVICE_FAULT"):
        s.cache.check()
    s.cache.check()  # reported once
    if what != "page":
        assert (out[:new] == -7.0).all()
    if what != "span":  # the second sequence is served
        n = s.lens[1]
        rows = R.quantised(k[new:].double().cpu().numpy())
        kk, vv = (x.copy() for x in kv[1])
        kk[n - new:], vv[n - new:] = rows, rows
        want, reach = R.attention(q[new:].double().cpu().numpy(), kk, vv, n, R.default_scale(64))
        err = np.abs(out[new:].double().cpu().numpy() - want)
        assert (err <= R.tolerance(want, reach, np.abs(vv).max(), "bf16")).all()


def test_refusals():
    from persistent_megakernel_02_b200 import Kv4Cache, MkError

    s = Setup(64, 2, [40], [40])
    q, k = s.rand(40, 8, "bf16"), s.rand(40, 2, "bf16")

    def refused(fn, *a, **kw):
        with pytest.raises(MkError, match="INVALID_ARG|UNSUPPORTED"):
            fn(*a, **kw)

    refused(s.cache.append, 1, k, k, s.batch)                         # layer
    refused(s.cache.append, 0, k.float(), k, s.batch)                 # two types
    refused(s.cache.append, 0, k.double(), k.double(), s.batch)
    refused(s.cache.append, 0, k[:39], k[:39], s.batch)               # rows
    refused(s.cache.append, 0, q, q, s.batch)                         # heads
    refused(s.cache.append, 0, k.cpu(), k.cpu(), s.batch)
    refused(s.cache.append, 0, k.transpose(0, 2), k, s.batch)
    flat = torch.zeros(40 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    refused(s.cache.append, 0, flat[1:].view(40, 2, 64), k, s.batch)  # not 16-byte aligned
    refused(s.cache.read, 0, k[:1].expand(40, 2, 64), k, s.batch)     # an output that overlaps itself
    refused(s.cache.read, 0, k, k, s.batch)                           # one output for both
    refused(s.cache.attend, 0, q, torch.empty_like(q).float(), s.batch)
    refused(s.cache.attend, 0, s.rand(40, 3, "bf16"), s.rand(40, 3, "bf16"), s.batch)
    refused(s.cache.attend, 0, s.rand(40, 32, "bf16"), s.rand(40, 32, "bf16"), s.batch)  # 16 per kv head
    refused(s.cache.attend, 0, q, torch.empty_like(q), s.batch, scale=float("nan"))
    refused(s.cache.attend, 0, q, torch.empty_like(q), s.batch, scale=3e38)
    refused(s.cache.attend, 0, q[:, :, ::2], torch.empty_like(q), s.batch)
    refused(Kv4Cache, s.cache.pool, s.table, 128)
    refused(Kv4Cache, s.cache.pool.cpu(), s.table, 64)
    refused(s.cache.batch, s.cu, s.kv_lens, 40, 40, 64 * s.table.shape[1] + 1)
    refused(s.cache.batch, s.cu[:1], s.kv_lens, 40, 40, 40)
    refused(s.cache.batch, s.cu.long(), s.kv_lens, 40, 40, 40)
    long = Setup(64, 8, [9000], [1])
    x = long.rand(1, 32, "bf16")
    if long.cache.workspace_bytes(long.batch, 32, torch.bfloat16):
        refused(long.cache.attend, 0, x, torch.empty_like(x), long.batch,
                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    s.cache.check()


def test_no_rows_and_no_new_rows():
    s = Setup(64, 2, [40], [0])
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    s.cache.append(0, none, none, s.batch)
    s.cache.read(0, none, none, s.batch)
    s.cache.attend(0, torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"),
                   torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), s.batch)
    s.cache.check()
    assert (s.pool() == 255).all()


# ---- with the framework's own paths ----------------------------------------------------


@pytest.mark.parametrize("kv_dtype", [0, 1])
def test_parked_sequence_decodes_after_it_comes_back(kv_dtype):
    """Prefill two slots, park both, let others use the slots, resume swapped, decode: the logits
    are the oracle's over the values the cache stands for."""
    from oracle import OracleModel, weights_to_numpy
    from persistent_megakernel_02_b200 import Kv4Cache, Megakernel

    cfg = configs.model_config("tiny", max_batch=2, max_seq=160, kv_dtype=kv_dtype)
    w = synth.make_weights(cfg, device="cuda")
    mk = Megakernel(cfg, w)
    lens = [131, 40]
    prompts = [synth.prompt_tokens(cfg, i, n).tolist() for i, n in enumerate(lens)]
    for i in range(2):
        mk.prefill(i, prompts[i])
    table = torch.tensor([[4, 1, 3], [2, 0, 0]], dtype=torch.int32, device="cuda")
    cache = Kv4Cache.empty(cfg["n_layers"], 5, cfg["n_kv_heads"], cfg["head_dim"], table)
    cache.pool.fill_(255)
    mk.park(0, lens[0], cache, 0)
    mk.park(1, 25, cache, 1)                # in two pieces
    mk.park(1, 15, cache, 1, start=25)
    other = synth.prompt_tokens(cfg, 7, 150).tolist()
    for i in range(2):
        mk.prefill(i, other)
    mk.resume(1, lens[0], cache, 0)
    mk.resume(0, 10, cache, 1)
    mk.resume(0, 30, cache, 1, start=10)
    mk.sync()
    cache.check()
    pool = cache.pool.cpu().numpy()
    orc = OracleModel(cfg, weights_to_numpy(w), np.float32, kv_round="fp16" if kv_dtype else "bf16")
    oracle_caches = []
    for seq, slot in ((1, 0), (0, 1)):
        oc = orc.new_cache()
        plain = orc.new_cache()
        for p, t in enumerate(prompts[seq]):
            orc.step(t, p, plain)
        for layer in range(cfg["n_layers"]):
            pages = table[seq].cpu().numpy()[: -(-lens[seq] // 64)]
            got = R.unpack(pool, layer, pages, lens[seq])
            for name, x in zip(("K", "V"), got):
                true = np.stack(plain[name][layer])
                _, step, _ = R.quantise(true.astype(np.float64))
                # half a step (of these values, up to their own error), plus the parity error of K and V
                bound = 0.5 * np.repeat(step, 32, -1) * 1.02 + 2e-2 * max(1.0, np.abs(true).max())
                assert (np.abs(x - true) <= bound).all()
                rounded = torch.from_numpy(x).float().to(torch.float16 if kv_dtype else torch.bfloat16).float().numpy()
                oc[name][layer] = [r for r in rounded]
        oracle_caches.append((seq, slot, oc))
    tok = torch.tensor([11, 23], dtype=torch.int32, device="cuda")
    ids = torch.empty(2, dtype=torch.int32, device="cuda")
    logits = torch.empty((2, cfg["vocab"]), dtype=torch.float32, device="cuda")
    mk.decode_step(tok, [lens[1], lens[0]], ids, logits)
    mk.sync()
    for seq, slot, oc in oracle_caches:
        want = orc.step(int(tok[slot]), lens[seq], oc)
        H.compare_logits(logits[slot].cpu().numpy(), want, f"slot {slot}")
    mk.close()


def test_park_refusals():
    from persistent_megakernel_02_b200 import Kv4Cache, Megakernel, MkError

    cfg = configs.model_config("tiny", max_batch=1, max_seq=100)
    mk = Megakernel(cfg, synth.make_weights(cfg, device="cuda"))
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    cache = Kv4Cache.empty(cfg["n_layers"], 2, cfg["n_kv_heads"], cfg["head_dim"], table)
    for bad in (dict(slot=1, n=5, seq=0), dict(slot=-1, n=5, seq=0), dict(slot=0, n=101, seq=0), dict(slot=0, n=-1, seq=0),
                dict(slot=0, n=5, seq=1), dict(slot=0, n=5, seq=-1), dict(slot=0, n=5, seq=0, start=-1),
                dict(slot=0, n=2, seq=0, start=99),
                dict(slot=0, n=65, seq=0, block_table=table[:, :1].contiguous()),
                dict(slot=0, n=5, seq=0, block_table=table.long())):
        for move in (mk.park, mk.resume):
            with pytest.raises(MkError, match="INVALID_ARG"):
                move(bad["slot"], bad["n"], cache, bad["seq"], start=bad.get("start", 0),
                     block_table=bad.get("block_table"))
    wrong = Kv4Cache.empty(cfg["n_layers"] + 1, 2, cfg["n_kv_heads"], cfg["head_dim"], table)
    with pytest.raises(MkError, match="INVALID_ARG"):
        mk.park(0, 5, wrong, 0)
    mk.park(0, 0, cache, 0)
    mk.sync()
    mk.close()


def test_a_decoder_step_from_the_stand_alone_stages():
    """One layer run by the caller: the streaming matvec for q, k, v and the output projection, the
    4-bit cache, the greedy head; against 64 bits over the values the cache stands for."""
    from persistent_megakernel_02_b200 import Kv4Cache, greedy_head_noalloc, matvec_engine, matvec_engine_status

    hidden, heads, kvh, d, nb, steps = 2048, 32, 8, 64, 3, 4
    wq, wk, wv, wo = (synth.normal_bf16(shape, 9, i, std=0.02, device="cuda") for i, shape in enumerate(
        ((heads * d, hidden), (kvh * d, hidden), (kvh * d, hidden), (hidden, heads * d))))
    lm = synth.normal_bf16((4096, hidden), 9, 5, std=0.02, device="cuda")
    gain = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(nb, dtype=torch.int32, device="cuda").view(nb, 1).contiguous()
    cache = Kv4Cache.empty(1, nb, kvh, d, table)
    cu = torch.arange(nb + 1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(nb, dtype=torch.int32, device="cuda")
    batch = cache.batch(cu, lens, nb, 1, 64)
    x = synth.normal_bf16((nb, hidden), 9, 6, std=1.0, device="cuda").float().contiguous()
    f64 = [w.double() for w in (wq, wk, wv, wo, lm)]
    past = [[], []]
    for step in range(steps):
        lens.fill_(step + 1)
        q, k, v = (torch.empty((nb, n * d), device="cuda") for n in (heads, kvh, kvh))
        o, y = torch.empty_like(q), torch.empty_like(x)
        for w, t in ((wq, q), (wk, k), (wv, v)):
            matvec_engine("cuda_cores", w, x, t)
        cache.append(0, k.view(nb, kvh, d), v.view(nb, kvh, d), batch)
        cache.attend(0, q.view(nb, heads, d), o.view(nb, heads, d), batch)
        matvec_engine("cuda_cores", wo, o, y)
        ids = torch.empty(nb, dtype=torch.int32, device="cuda")
        logits = torch.empty((nb, 4096), device="cuda")
        greedy_head_noalloc(y, gain, lm, 1e-5, ids, logits)
        matvec_engine_status()
        cache.check()
        for kept, t, w in zip(past, (k, v), f64[1:3]):
            assert torch.allclose(t.double(), x.double() @ w.T, atol=1e-4)
            kept.append(torch.from_numpy(R.quantised(t.double().cpu().numpy().reshape(nb, kvh, d))))
        qn = (x.double() @ f64[0].T).cpu().numpy().reshape(nb, heads, d)
        want_o = np.stack([R.attention(qn[b:b + 1], *(np.stack([r[b].numpy() for r in kept]) for kept in past),
                                       step + 1, R.default_scale(d))[0][0] for b in range(nb)])
        want = torch.from_numpy(want_o.reshape(nb, -1)).cuda() @ f64[3].T
        n = want / torch.sqrt((want * want).mean(-1, keepdim=True) + 1e-5)
        assert (logits.double() - n @ f64[4].T).abs().max() < 1e-3
        x = y  # the next step sees another state


@pytest.mark.parametrize("d,lens,new", [(64, [2000], [1]), (128, [900, 1500], [1, 1]), (64, [16384], [1]), (64, [600], [200])])
def test_32_bit_calls_keep_32_bits(d, lens, new):
    """The 2-norm of the error over that of the result.  Every part of the computation is good
    to 2^-21 of its terms, and the terms' signs vary: 2^-18 leaves a factor of 8 for the
    codes' and the minima's parts, which partly cancel.  Keys with large channels, as a
    decoder makes them."""
    s = Setup(d, 2, lens, new)
    kv = s.fill()
    q = s.rand(s.rows, 8, "fp32")
    out = torch.empty_like(q)
    s.cache.attend(0, q, out, s.batch)
    got = out.double().cpu().numpy()
    for i, (n_len, n) in enumerate(zip(lens, new)):
        a, b = s.cu_np[i], s.cu_np[i + 1]
        want, _ = R.attention(q[a:b].double().cpu().numpy(), *kv[i], n_len, R.default_scale(d))
        assert np.linalg.norm(got[a:b] - want) / np.linalg.norm(want) < 2.0**-18


@pytest.mark.parametrize("keys", [1.0, 8.0, 1e-5])
@pytest.mark.parametrize("d,kv_heads,lens,new", [(64, 16, [2000], [400]), (128, 16, [900, 70], [300, 70]), (64, 8, [700] * 3, [65, 200, 700]),
                                                 (128, 2, [3000], [150]), (64, 2, [5000], [1])])
def test_fp16_calls_round_only_the_weights(d, kv_heads, lens, new, keys):
    """The 2-norm of the error over that of the result.  Rounding to fp16 is off by u / m with u
    evenly spread up to 2^-11 and m the mantissa, 1 to 2: 2.1e-4 in the mean of squares over
    a binade.  Weights and outputs take one each, 2.9e-4 together, and mantissas not spread
    evenly an eighth more: 3.3e-4.  K and V are good to 2^-17 of their group's largest, which
    does not show, but for V of 128-value heads in prompts: a third rounding, 2.1e-4 x sqrt(3)
    and an eighth more, 4.1e-4.  K rounded to fp16 would make these 4.7e-4 to 6.8e-4."""
    s = Setup(d, kv_heads, lens, new)
    kv = s.fill(keys=keys)
    q = (s.rand(s.rows, 4 * kv_heads, "fp32") / keys).half()
    q = q if keys >= 1 else s.rand(s.rows, 4 * kv_heads, "fp16")
    out = torch.empty_like(q)
    scale = R.default_scale(d) * (1 if keys >= 1 else 1 / keys)
    s.cache.attend(0, q, out, s.batch, scale=scale)
    got = out.double().cpu().numpy()
    for i in range(len(lens)):
        a, b = s.cu_np[i], s.cu_np[i + 1]
        want, _ = reference(s, kv, q, i, scale)
        assert np.linalg.norm(got[a:b] - want) / np.linalg.norm(want) < (4.1e-4 if d == 128 else 3.3e-4)


@pytest.mark.parametrize("d,n_len", [(64, 131072 + 77), (128, 70000)])
def test_prompts_over_very_long_caches_keep_their_sums(d, n_len):
    """Values with a mean of 2, so that sums grow: the mean of the relative errors.  The output's
    rounding has no mean (16 x 8 x d of it, 2.1e-4 each: 1e-6 to 2e-6), a sum that is cut off
    has: at most 32768 positions are added up before the parts are joined, at 2^-27 each."""
    new, rep = 4800, 8  # enough blocks that nothing else splits the positions
    rng = np.random.default_rng(2)
    s = Setup(d, 1, [1], [1])
    table = torch.from_numpy(R.tables([n_len], rng)[0]).cuda()
    cache = type(s.cache).empty(1, int(table.shape[1]) + 2, 1, d, table)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((n_len, 1, d), device="cuda", generator=g) + x for x in (0.0, 2.0))
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n_len], [0, new], [n_len])]
    whole = cache.batch(ints[0], ints[2], n_len, n_len, n_len)
    cache.append(0, k, v, whole)
    cache.read(0, k, v, whole)
    batch = cache.batch(ints[1], ints[2], new, new, n_len)
    q = torch.randn((new, rep, d), device="cuda", generator=g).half()
    out = torch.empty_like(q)
    cache.attend(0, q, out, batch)
    cache.check()
    at = torch.arange(n_len, device="cuda")
    see = at[None, None, :] <= at[-16:][:, None, None]
    sc = torch.einsum("qhd,pd->qhp", q[-16:].double(), k[:, 0].double()) * R.default_scale(d)
    want = torch.einsum("qhp,pd->qhd", torch.softmax(sc.masked_fill(~see, -np.inf), -1), v[:, 0].double())
    off = (out[-16:].double() - want) / want
    assert off.mean().abs() < 32768 * 2.0**-27 + 4e-5 and off.abs().max() < 2.0**-9


@pytest.mark.parametrize("new", [1, 40, 700])
def test_pools_of_more_than_32_bits_of_bytes(new):
    """Pages and a layer behind 2^32 bytes, and rows whose strides lead there too."""
    from persistent_megakernel_02_b200 import Kv4Cache

    d, kvh, n_len = 128, 8, 900
    n_pages = 2**32 // (kvh * 64 * 20 * d // 16) + 50
    table = torch.arange(n_pages - 1, n_pages - 1 - 16, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    cache = Kv4Cache.empty(2, n_pages, kvh, d, table)
    s = Setup(d, kvh, [n_len], [new])
    s.table, s.cache = table, cache
    s.batch = cache.batch(s.cu, s.kv_lens, new, new, n_len)
    kv = s.fill(layer=1)
    far = torch.empty((2, 4 * kvh, 2**26 + d), dtype=torch.bfloat16, device="cuda")  # 128 MiB from head to head
    q, out = (far[i].as_strided((new, 4 * kvh, d), (d, 2**26 + d, 1), far[i].storage_offset()) for i in range(2))
    q.copy_(s.rand(new, 4 * kvh, "bf16"))
    cache.attend(1, q, out, s.batch)
    check_attention(s, kv, q.contiguous(), out.contiguous(), "bf16")
    k, v = (far[i].as_strided((new, kvh, d), (d, 2**26 + d, 1), far[i].storage_offset()) for i in range(2))
    cache.read(1, k, v, s.batch)
    cache.check()
    for t, x in zip((k, v), kv[0]):
        assert torch.equal(t.cpu(), torch.from_numpy(x[n_len - new:]).float().bfloat16())
