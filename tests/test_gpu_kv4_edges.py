"""The 4-bit KV cache on the GPU where a call can go wrong: long runs, far ranges, batches of very
unequal sequences, streams, errors (needs a B200)."""

import subprocess
import sys

import numpy as np
import pytest
import torch

import synth
from synth import configs
from tests import _kv4 as R
from tests.test_gpu_kv4 import Setup, check_attention, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from persistent_megakernel_02_b200 import build

    build.build()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Shared:
    """One sequence of `n_len` positions in a cache, and `lens` sequences that are its first positions:
    they read the same pages, so many long sequences cost one."""

    def __init__(self, d, kv_heads, n_len, lens, new=None, make_k=None, make_v=None, seed=0):
        from persistent_megakernel_02_b200 import Kv4Cache

        self.d, self.kv_heads, self.lens = d, kv_heads, list(lens)
        self.new = [1] * len(self.lens) if new is None else list(new)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        pages = -(-n_len // R.PAGE)
        row = torch.randperm(pages, generator=self.gen, device="cuda").int()
        self.table = row[None].expand(len(self.lens), pages).contiguous()
        self.cache = Kv4Cache.empty(1, pages, kv_heads, d, self.table)
        self.cache.pool.fill_(255)
        shape = (n_len, kv_heads, d)
        k, v = (torch.randn(shape, generator=self.gen, device="cuda") for _ in range(2))
        k, v = k if make_k is None else make_k(k), v if make_v is None else make_v(v)
        whole = self.cache.batch(ints([0, n_len]), ints([n_len]), n_len, n_len, n_len)
        self.cache.append(0, k, v, whole)
        self.cache.read(0, k, v, whole)  # what the cache stands for
        self.k, self.v = k, v
        self.cu = np.concatenate([[0], np.cumsum(self.new)])
        self.rows = int(self.cu[-1])
        self.batch = self.cache.batch(ints(self.cu), ints(self.lens), self.rows, max(self.new), max(self.lens))

    def queries(self, heads, dtype, size=1.0):
        return (torch.randn((self.rows, heads, self.d), generator=self.gen, device="cuda") * size).to(R.DTYPES[dtype])

    def attend(self, q, **kw):
        out = torch.full_like(q, -7.0)
        self.cache.attend(0, q, out, self.batch, **kw)
        return out

    def want(self, q, i, k=None, v=None, scale=None):
        """Rows of sequence i, float64."""
        k, v = self.k if k is None else k, self.v if v is None else v
        n, n_len = self.new[i], self.lens[i]
        x = q[self.cu[i]:self.cu[i + 1]].double()
        rep = q.shape[1] // self.kv_heads
        see = torch.arange(n_len, device="cuda")[None] <= torch.arange(n_len - n, n_len, device="cuda")[:, None]
        out = torch.empty_like(x)
        for h in range(q.shape[1]):
            kk, vv = k[:n_len, h // rep].double(), v[:n_len, h // rep].double()
            s = (x[:, h] @ kk.T * (R.default_scale(self.d) if scale is None else scale)).masked_fill(~see, -np.inf)
            out[:, h] = torch.softmax(s, -1) @ vv
        return out

    def got(self, out, i):
        return out[self.cu[i]:self.cu[i + 1]].double()


# Bounds of the 2-norm of the error over that of the result for single tokens and a few.  A rounding
# to t bits is off by u / m, u evenly spread up to half a step and m the mantissa, 1 to 2: in the mean
# of squares over a binade 2.1e-4 for fp16 and 1.67e-3 for bf16, and an eighth more for mantissas not
# spread evenly.
#   fp16: weights and outputs rounded, V as it is: 3.3e-4.
#   bf16: outputs rounded, weights and weight * scale to fp16.  The latter's part of a value, s c, is in
#   the mean of squares 2.3 times the value of normal rows (a group spans 4.1 of their deviations, so
#   codes stand for 2.05 +- 1 of them): sqrt(1.67^2 + 0.21^2 + 0.48^2) = 1.75e-3, and an eighth: 2.0e-3.
#   fp32: two fp16 parts of 22 bits, signs varying, a factor of 8 for the parts that cancel: 2^-18.
NORM = {"fp16": 3.3e-4, "bf16": 2.0e-3, "fp32": 2.0**-18}


def norm_error(got, want):
    return float(torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want))


# ---- sums over many positions -----------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,n_len", [(64, 131072 + 5), (64, 16384 + 37), (128, 65536 + 37), (128, 16384 + 1)])
def test_many_long_sequences_keep_their_sums(d, n_len, dtype):
    """So many sequences that nothing splits them but their length: a warp goes over thousands of
    positions, whose codes' and minima's parts largely cancel, so that a sum that is cut off, or
    that grows, shows.  Keys are small, as weights spread over many positions make it worst."""
    n = 150
    s = Shared(d, 8, n_len, [n_len - 61 * (i % 40) for i in range(n)], make_k=lambda k: k * 0.25)
    q = s.queries(16, dtype)
    out = s.attend(q)
    s.cache.check()
    for i in (0, 39, n - 1):
        want, got = s.want(q, i), s.got(out, i)
        assert norm_error(got, want) < NORM[dtype]
        # one head's row: 64 or 128 terms, half as much again
        worst = (torch.linalg.vector_norm(got - want, dim=-1) / torch.linalg.vector_norm(want, dim=-1)).max()
        assert float(worst) < 1.5 * NORM[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [2, 8])
def test_a_few_rows_of_many_long_sequences(d, new, dtype):
    n_len = 9000
    s = Shared(d, 8, n_len, [n_len - 61 * (i % 40) for i in range(80)], new=[new - i % 2 for i in range(80)],
               make_k=lambda k: k * 0.25)
    q = s.queries(32, dtype)
    out = s.attend(q)
    s.cache.check()
    for i in (0, 1, 39):
        assert norm_error(s.got(out, i), s.want(q, i)) < NORM[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (64, 4), (128, 4), (64, 40), (128, 40)])
def test_missing_pages_of_many_long_sequences(d, new, dtype):
    """Each page has values of its own and weights are nearly even, so a page that is left in or out
    wrongly moves the result by several per cent; pages far into a warp's run among them."""
    from persistent_megakernel_02_b200 import MkError

    n_len, gone = 9000, (0, 3, 31, 66, 67, 100, 131)
    pages = torch.randn((-(-n_len // 64), 8, d), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    spread = pages.repeat_interleave(64, 0)[:n_len]
    s = Shared(d, 8, n_len, [n_len - 7 * (i % 9) for i in range(90)], new=[new] * 90, make_k=lambda k: k * 0.1,
               make_v=lambda v: 0.2 * v + spread)
    q = s.queries(16, dtype)
    whole = s.want(q, 4)
    for i, page in enumerate(gone):
        s.table[:, page] = (-1, s.cache.n_pages, -2, 2**31 - 1)[i % 4]
    out = s.attend(q)
    with pytest.raises(MkError, match="a page id"):
        s.cache.check()
    keep = torch.ones(n_len, dtype=torch.bool, device="cuda")
    for page in gone:
        keep[64 * page:64 * page + 64] = False
    t = Shared.__new__(Shared)
    t.__dict__.update(s.__dict__)
    t.k, t.v, t.lens = s.k[keep], s.v[keep], [n - 64 * len(gone) for n in s.lens]
    for i in (0, 4, 89):
        # (of prompts K and V are rounded as well, one more of 2.1e-4 each)
        assert norm_error(s.got(out, i), t.want(q, i)) < (NORM[dtype] if new < 40 or dtype == "fp32" else NORM[dtype] + 2.4e-4)
    assert norm_error(s.got(out, 4), whole) > 0.03


# ---- a whole batch's bounds and a sequence's own ------------------------------------------


def mixed(d, kv_heads, lens, new, **kw):
    return Shared(d, kv_heads, max(lens), lens, new, make_k=lambda k: k * 0.25, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_workspace_of_a_mixed_batch_is_that_of_its_rows(dtype):
    """One long prompt beside single tokens, over caches long enough to be split."""
    from persistent_megakernel_02_b200 import Kv4Cache

    n, d, kvh, rep, prompt, top = 64, 128, 8, 4, 8192, 131072
    table = torch.zeros((n, top // 64), dtype=torch.int32, device="cuda")
    cache = Kv4Cache.empty(1, 1, kvh, d, table)
    cu = ints([0] + [prompt + i for i in range(n)])
    batch = cache.batch(cu, ints([top] * n), prompt + n - 1, prompt, top)
    # partial results: a row of D + 4 floats for every query row, head and split; 16 splits at most are
    # called for, and what a block of 256 rows is not filled by adds one block per sequence
    rows = (prompt + n) * rep + 256 * (n + 1)
    assert cache.workspace_bytes(batch, kvh * rep, R.DTYPES[dtype]) <= 16 * rows * kvh * (d + 4) * 4


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,kv_heads,lens,new", [
    (64, 8, [3000, 1500, 70, 2900, 1, 0, 2500] + [2999] * 20, [1500, 1, 3, 1, 1, 0, 700] + [1] * 20),
    (128, 8, [900] * 30 + [1100], [1] * 30 + [1100]),
    (64, 2, [5000, 4000, 3000], [65, 3000, 1]),
    (128, 8, [2000] + [1999] * 40, [1999] + [1] * 40),
    (64, 1, [40000, 100, 39000], [2049, 1, 300]),
])
def test_prompts_and_single_tokens_in_one_call(d, kv_heads, lens, new, dtype):
    s = mixed(d, kv_heads, lens, new)
    q = s.queries(4 * kv_heads, dtype)
    out = s.attend(q)
    s.cache.check()
    # rounding K and V in 16-bit prompts adds 2.1e-4 each, an eighth for uneven mantissas; rows that see
    # few positions, with weights far from even, are of the size of V, so the norm is over all
    bound = NORM[dtype] if dtype == "fp32" else NORM[dtype] + 2.4e-4
    for i in range(len(lens)):
        if new[i] and lens[i]:
            assert norm_error(s.got(out, i), s.want(q, i)) < bound, i
    again = s.attend(q)
    assert torch.equal(out, again)
    free = s.attend(q, workspace=torch.full((max(16, s.cache.workspace_bytes(s.batch, q.shape[1], q.dtype)),), 255,
                                            dtype=torch.uint8, device="cuda"))
    assert torch.equal(out, free)


@pytest.mark.parametrize("cu", [[0, 64, 0, 64], [0, 70, 30, 64], [0, 40, 10, 64], [64, 0, 64, 64], [0, 16, 17, 5],
                                [0, 64, 64, 0], [0, 10, 5, 5]])
@pytest.mark.parametrize("call", ["append", "read", "attend", "prompt"])
def test_a_cu_that_does_not_ascend_is_reported(cu, call):
    """... and a sequence is served as a whole or not at all; no two that are served share rows."""
    from persistent_megakernel_02_b200 import MkError

    s = Setup(64, 16, [200, 200, 200], [64, 64, 64])
    kv = s.fill()
    s.batch = s.cache.batch(ints(cu), s.kv_lens, 64, 64, 200)
    k, v = (s.rand(64, 16, "fp32") for _ in range(2))
    before = s.pool()
    if call == "append":
        s.cache.append(0, k, v, s.batch)
    elif call == "read":
        k.fill_(-7.0), v.fill_(-7.0)
        s.cache.read(0, k, v, s.batch)
    else:
        q = s.rand(64, 64, "fp32" if call == "attend" else "bf16")
        out = torch.full_like(q, -7.0)
        s.cache.attend(0, q, out, s.batch)
        assert torch.isfinite(out).all()
    with pytest.raises(MkError, match="batch numbers"):
        s.cache.check()
    s.cache.check()
    if call not in ("append", "read"):
        return
    after, taken = s.pool(), np.zeros(64, bool)
    for i in range(3):
        a, b = cu[i], cu[i + 1]
        got = R.unpack(after, 0, s.pages(i), 200)
        span = slice(200 - (b - a), 200) if b > a else slice(0, 0)
        if call == "append":
            if np.array_equal(after[:, s.pages(i)], before[:, s.pages(i)]):
                continue
            want = [x.copy() for x in kv[i]]
            for w, t in zip(want, (k, v)):
                w[span] = R.quantised(t[a:b].double().cpu().numpy())
            assert all(np.array_equal(w, g) for w, g in zip(want, got)), i
        else:
            rows = [x[span].astype(np.float32) for x in kv[i]]
            hit = [np.array_equal(t[a:b].cpu().numpy(), r) for t, r in zip((k, v), rows)] if b > a else [False]
            if not all(hit):
                continue
        assert 0 <= a < b <= 64 and not taken[a:b].any(), i
        taken[a:b] = True
    if call == "read":  # nothing else was written
        for t in (k, v):
            assert (t.cpu().numpy()[~taken] == -7.0).all()


@pytest.mark.parametrize("n", [31, 32, 33, 1000, 1025, 5000])
def test_batches_of_many_sequences(n):
    """Short sequences, some of them empty: every row finds its own."""
    rng = np.random.default_rng(n)
    new = rng.choice([0, 0, 1, 1, 2, 17, 33], n).tolist()
    lens = [v + int(x) for v, x in zip(new, rng.integers(0, 20, n))]
    s = Setup(64, 1, lens, new, pad_rows=5)
    k, v = s.rand(s.rows, 1, "bf16"), s.rand(s.rows, 1, "bf16")
    s.cache.append(0, k, v, s.batch)
    ko, vo = (torch.full_like(k, -7.0) for _ in range(2))
    s.cache.read(0, ko, vo, s.batch)
    s.cache.check()
    end = s.cu_np[-1]
    for t, o in ((k, ko), (v, vo)):
        want = torch.from_numpy(R.quantised(t[:end].double().cpu().numpy())).float().bfloat16()
        assert torch.equal(o[:end].cpu(), want) and (o[end:] == -7.0).all()


# ---- far ranges --------------------------------------------------------------------------


@pytest.mark.parametrize("new", [1, 300])
@pytest.mark.parametrize("d,kv_heads", [(64, 16), (128, 16)])
@pytest.mark.parametrize("dtype,q_size,scale", [
    ("bf16", 2.0**20, None), ("bf16", 2.0**23, None), ("bf16", 2.0**27, None), ("bf16", 2.0**60, None), ("bf16", 2.0**119, None),
    ("bf16", -(2.0**119), None), ("bf16", 1.0, 1e34), ("bf16", 1.0, -1e34), ("fp16", 1.0, 1e34), ("fp16", 40000.0, 2.0**10),
    ("fp32", 2.0**22, None), ("fp32", 2.0**27, None), ("fp32", 2.0**119, None), ("fp32", 1.0, 1e34),
])
def test_scores_far_from_each_other(dtype, q_size, scale, d, kv_heads, new):
    """Two positions with the same key far above the rest, all rows behind them: their mean, however
    large the finite scores are."""
    s = Setup(d, kv_heads, [900], [new])
    sign = torch.from_numpy(np.where(s.rng.random((1, kv_heads, d)) < 0.5, -1.0, 1.0)).float().cuda()
    up = sign if q_size * (1.0 if scale is None else scale) > 0 else -sign
    k, v = 0.1 * s.rand(900, kv_heads), s.rand(900, kv_heads)
    k[[5, 133]] = up * 2.0 * 64 / d
    s.cache.append(0, k, v, s.full_batch())
    v = torch.from_numpy(R.quantised(v.double().cpu().numpy()))
    q = (abs(q_size) * sign.repeat_interleave(2, 1).double() * (1 + 0.1 * torch.rand((new, 2 * kv_heads, d), device="cuda")))
    q = (q if q_size > 0 else -q).to(R.DTYPES[dtype])
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, q, out, s.batch, scale=scale)
    s.cache.check()
    want = ((v[5] + v[133]) / 2).repeat_interleave(2, 0)[None].numpy()
    err = np.abs(out.double().cpu().numpy() - want)
    # V, or weight and weight * scale, to fp16, and the output
    eps = torch.finfo(R.DTYPES[dtype]).eps / 2
    assert (err <= eps * np.abs(want) + np.abs(v.numpy()).max() * (2.0**-20 if dtype == "fp32" else 2.0**-10) + 2.0**-24).all()


@pytest.mark.parametrize("new", [1, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("q_size", [2.0**20, 2.0**25, 2.0**27, 2.0**90, 2.0**119])
def test_equal_scores_far_from_zero(q_size, dtype, new):
    """Keys that are all alike: the mean of the values, whatever the sign and size of the scores."""
    s = Setup(64, 16, [700], [new])
    k, v = s.rand(1, 16).expand(700, 16, 64), s.rand(700, 16)
    s.cache.append(0, k, v, s.full_batch())
    kv = [tuple(R.quantised(x.double().cpu().numpy()) for x in (k, v))]
    q = (s.rand(new, 32) * q_size).to(R.DTYPES[dtype])
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, q, out, s.batch)
    total = np.cumsum(kv[0][1], 0)
    see = np.arange(700 - new, 700)
    want = np.repeat(total[see] / (see + 1)[:, None, None], 2, 1)
    err = np.abs(out.double().cpu().numpy() - want)
    tol = R.tolerance(want, np.zeros(want.shape[:2]), np.abs(kv[0][1]).max(), dtype)
    assert (err <= tol).all(), f"{(err / tol).max()}"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("v_size", [2.0**-20, 2.0**-17, 2.0**-13, 2.0**-9, 1.0, 2.0**12])
@pytest.mark.parametrize("grow", [False, True])
def test_small_values_under_uneven_weights(v_size, d, dtype, grow):
    """Values whose scales are fp16's smallest, and a position in 200 with 2^12 times the others' weight:
    the others together still count.  `grow`: values 2^10 times as large come up later on."""
    n_len = 9000
    at = torch.rand(n_len, generator=torch.Generator("cuda").manual_seed(1), device="cuda") < 1 / 200

    def keys(k):
        k = torch.zeros_like(k)
        k[at] = 12.0 * np.log(2) / np.sqrt(d)  # with queries of ones: 12 in the exponent of 2
        return k

    def values(v):
        v = v * v_size
        if grow:
            v[5000:] *= min(2.0**10, 2.0**12 / v_size)
        return v

    s = Shared(d, 8, n_len, [4000 + 40 * (i % 120) for i in range(150)], make_k=keys, make_v=values)
    q = torch.ones((s.rows, 16, d), device="cuda").to(R.DTYPES[dtype])
    out = s.attend(q)
    s.cache.check()
    for i in (0, 24, 26, 119):
        assert norm_error(s.got(out, i), s.want(q, i)) < NORM[dtype], i


# ---- streams and errors --------------------------------------------------------------------


def tiny(**kw):
    from persistent_megakernel_02_b200 import Kv4Cache, Megakernel

    cfg = configs.model_config("tiny", max_batch=2, max_seq=160, **kw)
    mk = Megakernel(cfg, synth.make_weights(cfg, device="cuda"))
    table = ints([[4, 1, 3], [2, 0, 0]])
    return mk, cfg, Kv4Cache.empty(cfg["n_layers"], 5, cfg["n_kv_heads"], cfg["head_dim"], table)


@pytest.mark.parametrize("given", [False, True])
def test_park_and_resume_keep_the_order_of_the_current_stream(given):
    """The handle's steps run on the default stream unless told otherwise, the cache's calls on torch's
    current one: without a stream, park and resume come behind both and before what follows on either."""
    mk, cfg, cache = tiny()
    prompts = [synth.prompt_tokens(cfg, i, 130).tolist() for i in range(2)]
    shape = (130, cfg["n_kv_heads"], cfg["head_dim"])
    batch = cache.batch(ints([0, 130]), ints([130]), 130, 130, 130)
    want = []
    for i in range(2):  # what each prompt parks
        mk.prefill(0, prompts[i])
        mk.park(0, 130, cache, 0)
        kv = [torch.empty(shape, device="cuda") for _ in range(2)]
        cache.read(0, *kv, batch)
        torch.cuda.synchronize()
        want.append(kv)
    assert not torch.equal(want[0][0], want[1][0])
    side = torch.cuda.Stream()
    arg = {"stream": side} if given else {}
    slow = 200_000_000  # cycles, about 0.1 s
    # the handle's work is late: what is read on the current stream is the new prompt's all the same
    mk.prefill(0, prompts[0])
    mk.sync()
    cache.pool.zero_()
    torch.cuda.synchronize()
    got = [torch.empty(shape, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        if not given:
            with torch.cuda.stream(torch.cuda.default_stream()):
                torch.cuda._sleep(slow)
        mk.park(0, 130, cache, 0, **arg)
        cache.read(0, *got, batch)
        cache.check()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    # the cache's work is late: what is resumed is what the current stream writes
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(slow)
        for layer in range(cfg["n_layers"]):
            cache.append(layer, *want[1], batch)
        mk.resume(1, 130, cache, 0, **arg)
        cache.pool.zero_()  # behind the resume
        mk.park(1, 130, cache, 0, **arg)
        cache.read(0, *got, batch)
    torch.cuda.synchronize()
    # (what came out of a cache goes back into it within one more rounding to the handle's bf16, so
    # within one step of the grid; another prompt's values are far from that)
    for a, b in zip(got, want[1]):
        _, step, _ = R.quantise(b.double().cpu().numpy())
        assert (np.abs((a - b).double().cpu().numpy()) <= 1.1 * np.repeat(step, 32, -1) + 2.0**-7 * np.abs(b.cpu().numpy())).all()
    # a page that is missing is reported by a check on the current stream
    torch.cuda.synchronize()
    cache.block_table[0, 1] = 99
    torch.cuda.synchronize()
    from persistent_megakernel_02_b200 import MkError

    with torch.cuda.stream(side):
        if not given:
            with torch.cuda.stream(torch.cuda.default_stream()):
                torch.cuda._sleep(slow)
        mk.park(0, 130, cache, 0, **arg)
        with pytest.raises(MkError, match="a page id"):
            cache.check()
    torch.cuda.synchronize()
    mk.close()


def test_park_without_a_stream_inside_a_capture_is_refused():
    """The default stream cannot be captured; with the capturing stream the copy is captured and replays."""
    from persistent_megakernel_02_b200 import MkError

    mk, cfg, cache = tiny()
    mk.prefill(0, synth.prompt_tokens(cfg, 1, 100).tolist())
    mk.park(0, 100, cache, 0)
    mk.sync()
    want = cache.pool.clone()
    cache.pool.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(MkError, match="INVALID_ARG"):
            mk.park(0, 100, cache, 0)
        mk.park(0, 100, cache, 0, stream=torch.cuda.current_stream())
    cache.pool.zero_()
    graph.replay()
    torch.cuda.synchronize()
    pages = cache.block_table[0, :2].long()
    assert torch.equal(cache.pool[:, pages[0]], want[:, pages[0]])
    graph.reset()
    mk.close()


def test_no_report_is_lost_between_two_streams():
    """A call on one stream meets a bad page while a check runs on another: that check or the next
    one says so."""
    from persistent_megakernel_02_b200 import MkError

    s = Setup(64, 2, [40], [40])
    s.fill()
    q = s.rand(40, 8, "bf16")
    out = torch.empty_like(q)
    s.table[0, 0] = s.cache.n_pages
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def reported(stream):
        try:
            s.cache.check(stream=stream)
        except MkError:
            return True
        return False

    for i in range(1500):
        with torch.cuda.stream(one):
            torch.cuda._sleep(1000 + 97 * (i % 700))  # 1 to 36 us
        s.cache.attend(0, q, out, s.batch, stream=one)
        early = reported(two)
        assert reported(one) or early, i


def test_a_new_cache_may_be_used_on_any_stream_at_once():
    """Its status word is cleared before the constructor returns, also where its stream is busy."""
    from persistent_megakernel_02_b200 import Kv4Cache, MkError

    s = Setup(64, 2, [40], [40])
    q = s.rand(40, 8, "bf16")
    out = torch.empty_like(q)
    s.table[0, 0] = s.cache.n_pages
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    cache = Kv4Cache(s.cache.pool, s.table, 64)
    cache.attend(0, q, out, s.batch, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    with pytest.raises(MkError, match="a page id"):
        cache.check(stream=side)


PENDING = """
import sys, torch
sys.path.insert(0, %r)
from persistent_megakernel_02_b200 import MkError, greedy_head_noalloc, matvec_engine_status
from tests.test_gpu_kv4 import Setup, check_attention, reference
from tests.test_gpu_kv4_edges import tiny
sets = [Setup(64, 16, [700, 300], [1, 1]), Setup(64, 16, [700, 300], [300, 200]), Setup(64, 2, [9000], [1])]
for s in sets:
    s.fill()
mk, cfg, cache = tiny()
head = [torch.zeros((1, 64), device="cuda"), torch.zeros(64, dtype=torch.bfloat16, device="cuda"),
        torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")]
greedy_head_noalloc(*head, 1e-5, torch.zeros(1, dtype=torch.int32, device="cuda"))  # (its first call sets things up)
torch.cuda.synchronize()
try:  # waiting for a stream that is being captured is an error, which stays with the library's runtime
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        try:
            matvec_engine_status(torch.cuda.current_stream())
        except MkError:
            print("refused")
except Exception as e:
    print("capture ended")
torch.cuda.synchronize()
def refused(fn, *a):
    try:
        fn(*a)
        return False
    except MkError as e:
        return e.status == 4
before = cache.pool.clone()
for s in sets:
    pool = s.cache.pool.clone()
    q = torch.ones((s.rows, 4 * s.kv_heads, 64), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.full((s.rows, s.kv_heads, 64), 3.0, device="cuda") for _ in range(2))
    out = torch.full_like(q, -7.0)
    need = s.cache.workspace_bytes(s.batch, q.shape[1], q.dtype)  # (asks the device, launches nothing)
    assert refused(s.cache.append, 0, k, v, s.batch) and refused(s.cache.read, 0, k, v, s.batch)
    assert refused(s.cache.attend, 0, q, out, s.batch)
    torch.cuda.synchronize()
    assert (out == -7).all() and (k == 3).all() and (v == 3).all() and torch.equal(pool, s.cache.pool)
assert refused(mk.park, 0, 5, cache, 0) and refused(mk.resume, 0, 5, cache, 0)
torch.cuda.synchronize()
assert torch.equal(before, cache.pool)
try:
    greedy_head_noalloc(*head, 1e-5, torch.zeros(1, dtype=torch.int32, device="cuda"))
    print("error gone")
except MkError:
    print("error kept")
"""


def test_an_earlier_error_is_left_in_place():
    """An error that another call left pending is not these calls': they refuse, launch nothing and leave
    it, as the other stand-alone stages do."""
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", PENDING % root], capture_output=True, text=True, timeout=600, cwd=root)
    assert run.returncode == 0, run.stdout + run.stderr
    assert run.stdout.split("\n")[:3] == ["refused", "capture ended", "error kept"], run.stdout + run.stderr


# ---- inputs and bounds -----------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("new", [1, 3, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite_reach_only_their_rows(bad, new, dtype):
    s = Setup(64, 16, [700, 500, 400], [new] * 3)
    s.fill()
    q = s.rand(s.rows, 64, dtype)
    clean, out = torch.empty_like(q), torch.empty_like(q)
    s.cache.attend(0, q, clean, s.batch)
    hit = torch.zeros((s.rows, 64), dtype=torch.bool, device="cuda")
    for row, head, value in ((0, 0, 7), (s.rows - 1, 5, 0), (s.rows // 2, 63, 63)):
        q[row, head, value] = bad
        hit[row, head] = True
    s.cache.attend(0, q, out, s.batch)
    s.cache.check()
    assert not torch.isfinite(out[hit]).any()
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,kv_heads", [([1500, 900], [1, 1], 8), ([9000], [1], 2), ([300] * 40 + [700], [1] * 40 + [300], 8),
                                               ([600, 500], [257, 64], 16), ([64], [64], 1)])
def test_bounds_wider_than_the_batch(lens, new, kv_heads, dtype):
    """As a captured step has them: room for more rows, longer spans and lengths than there are."""
    s = Setup(64, kv_heads, lens, new)
    kv = s.fill()
    pad = 900
    table = torch.full((len(lens), 2048), -1, dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = s.table
    q = s.rand(s.rows + pad, 4 * kv_heads, dtype)
    k, v = (torch.full((s.rows + pad, kv_heads, 64), -7.0, dtype=q.dtype, device="cuda") for _ in range(2))
    for max_new, max_len in ((max(new), 131072), (s.rows + pad, 20000), (s.rows + pad, 131072)):
        batch = s.cache.batch(s.cu, s.kv_lens, s.rows + pad, max_new, max_len, block_table=table)
        out = torch.full_like(q, -7.0)
        s.cache.attend(0, q, out, batch)
        s.cache.read(0, k, v, batch)
        s.cache.check()
        for i, (n_len, n) in enumerate(zip(lens, new)):
            a, b = s.cu_np[i], s.cu_np[i + 1]
            want, _ = reference(s, kv, q, i, R.default_scale(64))
            want = torch.from_numpy(want).cuda()
            assert norm_error(out[a:b].double(), want) < (NORM[dtype] if dtype == "fp32" else NORM[dtype] + 2.4e-4)
            for t, x in ((k, kv[i][0]), (v, kv[i][1])):
                assert torch.equal(t[a:b].cpu(), torch.from_numpy(x[n_len - n:]).float().to(q.dtype))
        for t in (out, k, v):
            assert (t[s.rows:] == -7.0).all()


@pytest.mark.parametrize("new", [1, 300])
def test_broadcast_queries(new):
    """One query for all heads, or for all rows: strides of zero."""
    s = Setup(128, 16, [500, 400], [new, new])
    kv = s.fill()
    for q in (s.rand(s.rows, 1, "bf16").expand(s.rows, 32, 128), s.rand(1, 32, "bf16").expand(s.rows, 32, 128)):
        out = torch.empty((s.rows, 32, 128), dtype=torch.bfloat16, device="cuda")
        s.cache.attend(0, q, out, s.batch)
        check_attention(s, kv, q, out, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new", [1, 300])
@pytest.mark.parametrize("power", [-60, -100, -115, -122])
def test_tiny_queries_under_a_large_scale(power, new, dtype):
    """Queries of 2^power and a scale that takes that back: the same as queries of ordinary size."""
    s = Setup(64, 16, [700], [new])
    kv = s.fill()
    q = s.rand(new, 32, dtype)
    small = q * 2.0**power  # (the smallest of 2^-122 are subnormal)
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, small, out, s.batch, scale=2.0**(-power - 3))
    check_attention(s, kv, small.double() * 2.0**-power, out, dtype, 0.125)


@pytest.mark.parametrize("at", [1, 2, 5])
def test_a_cu_that_does_not_ascend_in_a_batch_packed_by_its_rows(at):
    """One prompt and single tokens, whose row tiles are found by a search: reported, and every sequence is
    right or as it was."""
    from persistent_megakernel_02_b200 import MkError

    new = [600] + [1] * 7
    lens = [700, 650, 300, 20, 500, 660, 70, 100]
    s = Setup(64, 8, lens, new)
    kv = s.fill()
    cu = s.cu_np.copy()
    cu[at] -= 20  # in front of the end of the sequence before, or (1) rows of the prompt's for the next one
    s.batch = s.cache.batch(ints(cu), s.kv_lens, s.rows, 600, 700)
    q = s.rand(s.rows, 32, "bf16")
    out = torch.full_like(q, -7.0)
    s.cache.attend(0, q, out, s.batch)
    if (np.diff(cu) < 0).any():
        with pytest.raises(MkError, match="batch numbers"):
            s.cache.check()
    s.cache.check()
    for i in range(8):
        a, b = cu[i], cu[i + 1]
        if a >= b or b - a > lens[i]:
            continue
        t = Setup.__new__(Setup)
        t.__dict__.update(s.__dict__)
        t.cu_np, t.new = cu, [max(0, int(cu[j + 1] - cu[j])) for j in range(8)]
        want = torch.from_numpy(reference(t, kv, q, i, R.default_scale(64))[0]).cuda()
        whole = norm_error(out[a:b].double(), want) < NORM["bf16"] + 2.4e-4
        others = [j for j in range(8) if j != i and cu[j] < b and cu[j + 1] > a]  # share rows with it
        assert whole or (out[a:b] == -7.0).all() or others, i
