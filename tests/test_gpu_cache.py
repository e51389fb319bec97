"""GPU parity of the 8-bit key/value cache (append, read, attention) against the float64 oracle.

Tolerances. Codes, scales and read values are equal: both sides round the same float64 quantities (a quantity
within 1e-13 of a rounding border would be the exception; the seeded inputs hold none). Rotated queries: one
rounding, 2^-24 relative for float32 (and 1e-13 of the row for the float64 steps), 2^-8 + 2^-24 for bf16.

Attention, with S = scale max_t sum_d |q_d k_td|, V = sum_t p_t |v_t| per output entry, T the tokens seen:
  score error (base e): S (2^-22 [two float16 pieces of a float32 q; 0 for bf16] + (D + 8) 2^-24 [float32 sums,
  the scale factors, the fused multiply-add]) + 2^-18 [exponents up to 64 in float32: half a unit of 2^-17 in base 2]
  weight error eps: that + 2^-22 [exp2, reciprocal and logarithm, a few units] + 2^-21 [two pieces, float32] or
  2^-11 [one, bf16]
  output error: V (2 eps + (T + 32) 2^-24 [float32 sums of weights and products, joins]) + 2^-24 |out| (float32) or
  2^-8 |out| (bf16), and 127 T 2^-39 max_t p_t s_v,t: a weight is taken relative to the largest p_t s_v,t and goes to
  float16 times 2^14, whose smallest step is 2^-24, so each of the T weights is off by up to 2^-25 2^-14 of that largest
  one whatever its own size, times a code of up to 127. It counts where the heavy tokens' codes of a channel are 0, so
  that V is far below max p s_v (the rule above holds relative to V alone only while weights stay normal numbers).
"""
import numpy as np
import pytest

from gpu_helpers import DEV, host, require_gpu, to_dev
from oracle import kvcache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _kq():
    import post_quantization_04_amd as kq
    return kq


def _bf16(x):
    """float64 -> the nearest bf16 values, as float32."""
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def _dev(x, dtype):
    import torch
    return to_dev(np.asarray(x, np.float32), torch.bfloat16 if dtype == "bf16" else None)


def upload(cache):
    kq = _kq()
    return kq.KVCache(*(to_dev(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def batch_of(table, lens, q_start, max_q=None):
    kq = _kq()
    n = max([b - a for a, b in zip(q_start[:-1], q_start[1:])] + [1])
    return kq.CacheBatch(*(to_dev(np.asarray(t, np.int32)) for t in (table, lens, q_start)), n if max_q is None else max_q)


def tables(rng, lens, page, spare=2):
    """Scattered pages for each sequence; entries past a sequence's last page are no pages."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    order = rng.permutation(pages)[:sum(counts)]
    table = np.full((len(lens), max(max(counts), 1)), -7, np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, pages


def filled(rng, pages, page, kvh, dim, spread=0.3):
    c = kvcache.Cache.zeros(pages, page, kvh, dim)
    c.k[:] = np.clip(np.rint(rng.standard_normal(c.k.shape) * 38), -127, 127)
    c.v[:] = np.clip(np.rint(rng.standard_normal(c.v.shape) * 38), -127, 127)
    c.k_scale[:] = 0.025 * np.exp(spread * rng.standard_normal(c.k_scale.shape))
    c.v_scale[:] = 0.01 * np.exp(spread * rng.standard_normal(c.v_scale.shape))
    return c


def check_cache(dev, want, label=""):
    for name in ("k_scale", "v_scale", "k", "v"):
        np.testing.assert_array_equal(host(getattr(dev, name)), getattr(want, name), err_msg=f"{label} {name}")


def check_q(got, want, dtype):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    rel = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8 + 2.0 ** -24
    tol = rel * np.abs(want) + 1e-13 * np.max(np.abs(want), axis=-1, keepdims=True)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)


# ---- append -----------------------------------------------------------------------------------------------------


def append_case(seed, dtype, heads, kvh, dim, page, lens, news, *, norm=False, rot=None, inter=False, in_place=False,
                with_q=True, strided=True):
    import torch
    kq = _kq()
    from post_quantization_04_amd import pipeline
    rng = np.random.default_rng(seed)
    print(f"append {dtype} heads={heads}/{kvh} dim={dim} page={page} lens={lens} news={news} norm={norm} rot={rot} "
          f"inter={inter}", flush=True)
    table, pages = tables(rng, lens, page)
    want = filled(rng, pages, page, kvh, dim)
    q_start = np.concatenate(([0], np.cumsum(news)))
    rows = int(q_start[-1]) + 2                      # two rows behind the last sequence
    wide = (heads if with_q else 0) + 2 * kvh
    x = rng.standard_normal((rows, wide, dim)) * np.exp(rng.standard_normal(dim) * 0.7)
    x = _bf16(x) if dtype == "bf16" else x.astype(np.float32)
    xd = _dev(x, dtype)
    if not strided:
        xd = xd.clone()
    hq = heads if with_q else 0
    q, k, v = (xd[:, :hq], xd[:, hq:hq + kvh], xd[:, hq + kvh:])
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw = (1 + 0.1 * rng.standard_normal(dim)).astype(np.float32) if norm else None
    kw = (1 + 0.1 * rng.standard_normal(dim)).astype(np.float32) if norm else None
    rope = None if rot == 0 else pipeline.rope_table(max(max(lens), 1), dim if rot is None else rot)
    out = None
    if with_q:
        out = q if in_place else torch.full((rows, heads, dim), 3.0, dtype=xd.dtype, device=DEV)
    dev = upload(want)
    b = batch_of(table, lens, q_start)
    info = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = lambda: kq.cache_append(dev, b, q if with_q else None, k, v, out, q_norm=None if qw is None else to_dev(qw),  # noqa: E731
                                   k_norm=None if kw is None else to_dev(kw), eps=1e-5,
                                   rope=None if rope is None else rope.to(DEV), interleaved=inter, info=info)
    call()
    x64 = x.astype(np.float64)
    want_q = kvcache.append(want, table, lens, q_start, x64[:, :hq] if with_q else None, x64[:, hq:hq + kvh], x64[:, hq + kvh:],
                            q_norm=qw, k_norm=kw, eps=1e-5, rope=None if rope is None else rope.numpy(), interleaved=inter)
    check_cache(dev, want)
    assert int(info.item()) == 0
    if with_q:
        n = int(q_start[-1])
        if n:
            check_q(out[:n].float().cpu().numpy(), want_q[:n], dtype)
        tail = x[n:, :heads] if in_place else np.full((2, heads, dim), 3.0)
        np.testing.assert_array_equal(out[n:].float().cpu().numpy(), tail)
    if not in_place:
        call()  # the same tokens again: nothing left to change
        check_cache(dev, want, "again")
    return dev, want, table


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_tokens_and_prompts(dtype, dim, page):
    # single tokens at the first, a middle and the last slot of a page and of a 16-token group; prompts that begin and
    # end inside pages; a sequence without new tokens; an empty one
    lens = [1, page, page + 1, 2 * page - 5, 16, 17, 3 * page + 2, 2 * page, page + 9, 7, 0, 200]
    news = [1, 1, 1, 1, 1, 1, 2 * page + 5, 2 * page, 3, 0, 0, 190]
    append_case(page + dim, dtype, 4, 2, dim, page, lens, news)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kvh,dim,rot,inter,norm", [
    (3, 1, 128, 128, True, False), (6, 3, 128, 64, False, True), (5, 5, 64, 64, True, True), (8, 2, 64, 32, False, True),
    (1, 1, 128, 4, False, False), (2, 2, 64, 12, True, False), (9, 3, 128, 124, False, True), (4, 4, 64, 0, False, True),
    (7, 7, 128, 0, False, False)])
def test_append_norms_and_rotations(dtype, heads, kvh, dim, rot, inter, norm):
    append_case(heads * 100 + rot, dtype, heads, kvh, dim, 32, [45, 1, 64], [40, 1, 1], norm=norm, rot=rot, inter=inter)


def test_append_in_place_without_q_and_contiguous():
    append_case(1, "f32", 4, 2, 128, 16, [40, 3], [25, 1], in_place=True)
    append_case(2, "bf16", 4, 2, 64, 64, [40, 3], [25, 1], in_place=True, norm=True)
    append_case(3, "f32", 4, 2, 128, 16, [40, 3], [25, 1], with_q=False)
    append_case(4, "bf16", 4, 2, 128, 64, [400, 129], [300, 1], strided=False)
    append_case(5, "f32", 1, 1, 128, 64, [70], [1], strided=False)


def test_append_many_heads_of_a_long_prompt():
    # more than 8192 query rows: eight heads a wave, a last group of fewer
    append_case(6, "bf16", 13, 1, 64, 128, [700], [700])
    append_case(7, "f32", 13, 1, 128, 16, [650], [640], norm=True)


def test_append_growing_blocks():
    """A block filled token by token: every growth of its scale requantizes what is there."""
    import torch
    kq = _kq()
    rng = np.random.default_rng(9)
    for dim, page in ((128, 64), (64, 16), (128, 128)):
        want = kvcache.Cache.zeros(3, page, 2, dim)
        dev = upload(want)
        table = np.array([[2, 0]], np.int32)
        size = np.exp(np.cumsum(rng.standard_normal(page + 3) * 0.4))
        for t in range(page + 3):
            x = (rng.standard_normal((1, 4, dim)) * size[t]).astype(np.float32)
            if t == 5:
                x[:] = 0
            xd = to_dev(x)
            kq.cache_append(dev, batch_of(table, [t + 1], [0, 1]), None, xd[:, :2], xd[:, 2:])
            kvcache.append(want, table, [t + 1], [0, 1], None, x[:, :2].astype(np.float64), x[:, 2:].astype(np.float64))
        check_cache(dev, want, f"dim {dim} page {page}")
        torch.cuda.synchronize()


def test_append_extreme_values():
    """Zeros, values whose scale is at its floor, the largest, exact halves of a step, NaN and infinities: a bad
    entry marks its own block and head alone, for good."""
    kq = _kq()
    page, dim = 16, 64
    rng = np.random.default_rng(10)
    x = rng.standard_normal((40, 2, dim)).astype(np.float32)
    x[0:16] = 0                       # a block of zeros
    x[16:32, 0] *= 1e-36              # scale at its floor
    x[16:32, 1] *= 1e36
    x[16, 1, 0] = 3.4028234e38
    x[32:, 0] = rng.integers(-127, 128, (8, dim)) + 0.5
    x[32, 0, 0] = 127.0
    x[32:, 0] = np.clip(x[32:, 0], -127, 127)
    v = rng.standard_normal((40, 2, dim)).astype(np.float32)
    v[3, 1, 7] = np.nan
    v[17, 0, 0] = np.inf
    v[33, 1, 63] = -np.inf
    want = kvcache.Cache.zeros(3, page, 2, dim)
    dev = upload(want)
    table = np.array([[1, 2, 0]], np.int32)
    kq.cache_append(dev, batch_of(table, [40], [0, 40]), None, to_dev(x), to_dev(v))
    kvcache.append(want, table, [40], [0, 40], None, x.astype(np.float64), v.astype(np.float64))
    check_cache(dev, want)
    # what a block is given after a NaN does not mend it
    y = rng.standard_normal((1, 2, dim)).astype(np.float32)
    kq.cache_append(dev, batch_of(table, [41], [0, 1]), None, to_dev(y), to_dev(y))
    kvcache.append(want, table, [41], [0, 1], None, y.astype(np.float64), y.astype(np.float64))
    check_cache(dev, want, "after")
    assert np.isnan(want.v_scale[0, 1]) and not np.isnan(want.v_scale[0, 0])


def test_append_wrong_entries_are_told_and_not_followed():
    import torch
    kq = _kq()
    rng = np.random.default_rng(11)
    page, dim = 16, 64
    base = filled(rng, 4, page, 1, dim)

    def run(table, lens, q_start, rows=20, max_q=20, rope=None, q=True):
        x = rng.standard_normal((rows, 3, dim)).astype(np.float32)
        dev, xd = upload(base), to_dev(x)
        info = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full((rows, 1, dim), 5.0, device=DEV)
        kq.cache_append(dev, batch_of(table, lens, q_start, max_q), xd[:, :1], xd[:, 1:2], xd[:, 2:], out,
                        rope=None if rope is None else to_dev(rope), info=info)
        return dev, x.astype(np.float64), host(out), int(info.item())

    # a page that does not exist: its tokens are not stored, the others are
    for bad in (4, -1, 2 ** 31 - 1, -2 ** 31):
        dev, x, _, info = run([[1, bad, 2]], [40], [0, 20])
        want = base.copy()
        kvcache.append(want, [[1, bad, 2]], [40], [0, 20], None, x[:, 1:2], x[:, 2:])
        assert info == kq.KQ_INFO_PAGE
        check_cache(dev, want, f"page {bad}")
    # lengths: negative, past the table, fewer tokens than rows
    for length in (-5, -2 ** 31):
        dev, x, _, info = run([[1, 0, 2]], [length], [0, 20])
        assert info & kq.KQ_INFO_LENGTH
        check_cache(dev, base)
    dev, x, _, info = run([[1, 0, 2]], [2 ** 31 - 1], [0, 20])
    want = base.copy()
    kvcache.append(want, [[1, 0, 2]], [48], [0, 20], None, x[:, 1:2], x[:, 2:])
    assert info == kq.KQ_INFO_LENGTH
    check_cache(dev, want)
    dev, x, out, info = run([[1, 0, 2]], [7], [0, 20])
    want = base.copy()
    want_q = kvcache.append(want, [[1, 0, 2]], [7], [0, 20], x[:, :1], x[:, 1:2], x[:, 2:])
    assert info == kq.KQ_INFO_LENGTH
    check_cache(dev, want)
    assert np.isnan(out[:13]).all()
    check_q(out[13:], want_q[13:], "f32")
    # row ranges: past the rows, falling, more than max_q
    for q_start in ([0, 21], [-3, 20], [15, 5]):
        dev, _, _, info = run([[1, 0, 2]], [40], q_start)
        assert info & kq.KQ_INFO_ROWS
    dev, _, _, info = run([[1, 0, 2]], [40], [0, 20], max_q=7)
    assert info & kq.KQ_INFO_ROWS
    # a position past the rotations: NaN in q and in the block
    rope = np.concatenate((np.ones((30, 2)), np.zeros((30, 2))), 1).astype(np.float32)
    dev, x, out, info = run([[1, 0, 2]], [40], [0, 20], rope=rope)
    want = base.copy()
    want_q = kvcache.append(want, [[1, 0, 2]], [40], [0, 20], x[:, :1], x[:, 1:2], x[:, 2:], rope=rope)
    assert info == kq.KQ_INFO_POSITION
    check_cache(dev, want)
    assert np.isnan(out[10:]).all()
    check_q(out[:10], want_q[:10], "f32")


# ---- read -------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page,kvh", [(64, 16, 3), (128, 64, 2), (64, 128, 1), (128, 16, 5), (128, 32, 1)])
def test_read(dtype, dim, page, kvh):
    import torch
    kq = _kq()
    rng = np.random.default_rng(dim + page)
    lens, news = [1, 16, 100, 33, 0, 129, 64], [1, 16, 37, 0, 0, 129, 1]
    table, pages = tables(rng, lens, page)
    cache = filled(rng, pages, page, kvh, dim)
    q_start = np.concatenate(([0], np.cumsum(news)))
    rows = int(q_start[-1])
    dev = upload(cache)
    b = batch_of(table, lens, q_start)
    want = [np.concatenate([kvcache.tokens(cache, table[i], lens[i] - news[i], lens[i])[s] for i in range(len(lens))])
            .astype(np.float32) for s in (0, 1)]   # an 8-bit code times a 24-bit scale, rounded once
    if dtype == "bf16":
        want = [_bf16(w) for w in want]
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    both = torch.full((rows + 3, 2 * kvh, dim), 7.0, dtype=td, device=DEV)
    info = torch.zeros(1, dtype=torch.int32, device=DEV)
    kq.cache_read(dev, b, both[:, :kvh], both[:, kvh:], info=info)
    got = both.float().cpu().numpy()
    np.testing.assert_array_equal(got[:rows, :kvh], want[0])
    np.testing.assert_array_equal(got[:rows, kvh:], want[1])
    assert (got[rows:] == 7.0).all() and int(info.item()) == 0
    one = torch.full((rows, kvh, dim), 7.0, dtype=td, device=DEV)
    kq.cache_read(dev, b, one, None)
    np.testing.assert_array_equal(one.float().cpu().numpy(), want[0])
    kq.cache_read(dev, b, None, one)
    np.testing.assert_array_equal(one.float().cpu().numpy(), want[1])


def test_read_bad_pages_and_lengths():
    import torch
    kq = _kq()
    rng = np.random.default_rng(3)
    cache = filled(rng, 4, 16, 1, 64)
    dev = upload(cache)
    for table, n, bad in (([[0, 9, 2]], 40, kq.KQ_INFO_PAGE), ([[0, 1, 2]], 50, kq.KQ_INFO_LENGTH)):
        k, v = (torch.full((n, 1, 64), 7.0, device=DEV) for _ in range(2))
        info = torch.zeros(1, dtype=torch.int32, device=DEV)
        kq.cache_read(dev, batch_of(table, [40], [0, n]), k, v, info=info)
        wk, wv = kvcache.tokens(cache, table[0], 0, 40)
        pad = np.full((n - 40, 1, 64), np.nan)
        np.testing.assert_array_equal(host(k), np.concatenate((pad, wk)).astype(np.float32))
        np.testing.assert_array_equal(host(v), np.concatenate((pad, wv)).astype(np.float32))
        assert int(info.item()) == bad


# ---- attention --------------------------------------------------------------------------------------------------


def attention_tolerance(want, vabs, smax, top, seen, dim, dtype):
    score = smax * ((2.0 ** -22 if dtype == "f32" else 0.0) + (dim + 8) * 2.0 ** -24) + 2.0 ** -18
    eps = score + 2.0 ** -22 + (2.0 ** -21 if dtype == "f32" else 2.0 ** -11)
    out = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    return (vabs * (2 * eps[..., None] + (seen[:, None, None] + 32) * 2.0 ** -24) + out * np.abs(want)
            + 127 * 2.0 ** -39 * (seen[:, None] * top)[..., None])


def check_attention(got, cache, table, lens, q_start, q, scale, window, dtype):
    n = int(q_start[-1])
    if n == 0:
        return
    want, vabs, smax, top = kvcache.attention(cache, table, lens, q_start, q.astype(np.float64), scale, window)
    seen = np.concatenate([np.clip(lens[b] - (q_start[b + 1] - q_start[b]) + np.arange(q_start[b + 1] - q_start[b]) + 1, 0,
                                   window or None) for b in range(len(lens))]).astype(np.float64)
    got, want, vabs, smax, top = np.asarray(got, np.float64)[:n], want[:n], vabs[:n], smax[:n], top[:n]
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    tol = attention_tolerance(want, vabs, smax, top, seen, q.shape[2], dtype)
    off = np.abs(got - want)[fine] - tol[fine]
    assert off.size == 0 or np.max(off) <= 0, (np.max(off), np.max(np.abs(got - want)[fine]))
    if dtype == "bf16" and fine.any():  # far inside the worst case as a whole: output rounding plus the weights'
        norm = np.linalg.norm((got - want)[fine]) / max(np.linalg.norm(want[fine]), 1e-30)
        assert norm <= 2.0 ** -8


def attention_case(seed, dtype, heads, kvh, dim, page, lens, news, *, window=0, scale=None, spread=0.3, q_size=1.0,
                   max_q=None, cache=None, table=None, q=None, ws=True):
    import torch
    kq = _kq()
    rng = np.random.default_rng(seed)
    print(f"attention {dtype} heads={heads}/{kvh} dim={dim} page={page} lens={lens} news={news} window={window}", flush=True)
    if table is None:
        table, pages = tables(rng, lens, page)
    if cache is None:
        cache = filled(rng, pages, page, kvh, dim, spread)
    q_start = np.concatenate(([0], np.cumsum(news)))
    rows = int(q_start[-1]) + 2
    if q is None:
        q = rng.standard_normal((rows, heads, dim)) * q_size
    q = _bf16(q) if dtype == "bf16" else q.astype(np.float32)
    scale = dim ** -0.5 if scale is None else scale
    qd = _dev(np.concatenate((q, q[:, :1]), 1), dtype)[:, :heads]      # a pitch of its own
    dev = upload(cache)
    told = set()
    # the kernel goes by the bound on the rows of a sequence: as given, with the first one that takes the prompts' kernel
    # (few workgroups, so a long context is split there too), and with one that fills the GPU
    first = max(max(news), -(-max(16 * (256 // (len(lens) * kvh) + 1), 65) // (heads // kvh)))
    for bound in (max_q, first, 8192):
        if bound is not None and bound > rows:   # the bound counts up to the call's rows: more of them, of no sequence
            qd = torch.cat((qd, torch.full((bound - rows, heads, dim), float("nan"), dtype=qd.dtype, device=DEV)))
            rows = bound
        out = torch.full((rows, heads + 1, dim), 9.0, dtype=qd.dtype, device=DEV)[:, :heads]
        info = torch.zeros(1, dtype=torch.int32, device=DEV)
        b = batch_of(table, lens, q_start, bound)
        w = kq.cache_attention_workspace(dev, b, qd) if ws else None
        if w is not None and w.numel():
            w.fill_(255)                                               # NaN wherever it is read before it is written
        kq.cache_attention(dev, b, qd, out, scale=scale, window=window, info=info, ws=w)
        assert bool((out[int(q_start[-1]):] == 9.0).all())
        got = out[:int(q_start[-1]) + 2].float().cpu().numpy()
        check_attention(got, cache, table, lens, q_start, q, scale, window, dtype)
        told.add(int(info.item()))
    assert len(told) == 1
    return got, told.pop()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kvh,dim,page", [(4, 4, 128, 64), (8, 2, 128, 16), (5, 1, 64, 32), (16, 1, 128, 128),
                                                (14, 2, 64, 16), (40, 1, 128, 64), (6, 2, 64, 128)])
def test_attention_single_tokens(dtype, heads, kvh, dim, page):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 0, 511, 700]
    news = [1] * len(lens)
    news[2] = 0
    _, info = attention_case(heads + dim, dtype, heads, kvh, dim, page, lens, news)
    assert info == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
def test_attention_long_context_is_split(dtype, dim, page):
    """One sequence of thousands of tokens: many workgroups, joined; next to it short and empty ones."""
    attention_case(5, dtype, 8, 2, dim, page, [5003], [1])
    attention_case(6, dtype, 4, 1, dim, page, [3001, 1, 0, 70], [2, 1, 0, 3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kvh,dim,page,lens,news", [
    (4, 1, 128, 64, [5, 64, 100], [5, 64, 33]),
    (8, 2, 64, 16, [130, 1, 300], [130, 1, 17]),
    (3, 3, 128, 16, [257], [200]),
    (6, 2, 128, 128, [129, 260], [129, 255]),
    (8, 1, 64, 32, [400, 80], [70, 80]),
    (2, 2, 64, 64, [700], [650]),
    (12, 4, 128, 32, [333, 31, 64, 65], [300, 31, 64, 1]),
])
def test_attention_prompts(dtype, heads, kvh, dim, page, lens, news):
    _, info = attention_case(sum(lens), dtype, heads, kvh, dim, page, lens, news)
    assert info == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads,kvh,dim,page,length,new,window", [
    (16, 4, 128, 16, 300, 300, 0), (16, 4, 64, 64, 417, 289, 0), (8, 8, 128, 32, 700, 650, 90), (6, 6, 64, 16, 1100, 1100, 0),
    (16, 4, 128, 128, 250, 270, 33),
])
def test_attention_prompt_tiles(dtype, wide, heads, kvh, dim, page, length, new, window):
    """Few workgroups: in a table that holds little more than the prompt, rows in tiles of 128 with two waves for each 32;
    in one that could hold a long context before it, tiles of 256, split. The last case has rows without a token."""
    rng = np.random.default_rng(length)
    table, pages = tables(rng, [length], page)
    if wide:
        table = np.concatenate((table, np.full((1, 4 * new // page + 1), -7, np.int32)), 1)
    _, info = attention_case(new, dtype, heads, kvh, dim, page, [length], [new], window=window, table=table,
                             cache=filled(rng, pages, page, kvh, dim))
    assert info == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 300, 2 ** 31 - 1])
def test_attention_window(dtype, window):
    attention_case(window % 97, dtype, 8, 2, 128, 16, [1, 40, 333, 500], [1, 1, 3, 1], window=window)
    attention_case(window % 89, dtype, 4, 2, 64, 64, [300, 450], [290, 130], window=window)


def test_attention_pages_behind_the_window_are_not_looked_up():
    """A serving loop gives pages behind the window away: their table entries are no pages any more."""
    for news, heads in (([1], 4), ([90], 4), ([5], 4)):
        rng = np.random.default_rng(2)
        table, pages = tables(rng, [400], 16)
        cache = filled(rng, pages, 16, 1, 64)
        low = 400 - news[0] + 1 - 50
        table[0, :low // 16] = -1
        _, info = attention_case(3, "f32", heads, 1, 64, 16, [400], news, window=50, cache=cache, table=table)
        assert info == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_rows_without_a_token(dtype):
    """More rows than tokens in the cache: rows at negative positions see nothing and become zero."""
    for news in ([3, 4], [70, 90]):
        got, info = attention_case(7, dtype, 4, 2, 128, 16, [2, 0], news)
        assert info == 0
        assert not got[:news[0] - 2].any() and not got[news[0]:news[0] + news[1]].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [[1], [100]])
def test_attention_block_scales_far_apart(dtype, news):
    """Value scales from 2^-20 to 2^20 of each other, blocks of zeros among keys and values, peaked and flat rows."""
    rng = np.random.default_rng(4)
    table, pages = tables(rng, [300], 16)
    cache = filled(rng, pages, 16, 2, 64)
    cache.v_scale *= np.exp2(rng.uniform(-10, 10, cache.v_scale.shape)).astype(np.float32)
    for pg in table[0][[0, 5, 11]]:
        cache.v[pg], cache.v_scale[pg] = 0, 0.0
    for pg in table[0][[3, 5]]:
        cache.k[pg], cache.k_scale[pg] = 0, 0.0
    for size in (0.0, 1e-3, 1.0, 6.0):
        attention_case(5, dtype, 4, 2, 64, 16, [300], news, cache=cache, table=table, q_size=size)
    # all values zero
    cache.v[:], cache.v_scale[:] = 0, 0.0
    got, _ = attention_case(5, dtype, 4, 2, 64, 16, [300], news, cache=cache, table=table)
    assert not got[:news[0]].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [[1, 2], [60, 90]])
def test_attention_query_sizes(dtype, news):
    """Rows of zeros, of tiny and of huge entries (with a scale to match), and a row with a NaN or an infinity: that
    row alone is NaN."""
    rng = np.random.default_rng(6)
    rows = sum(news) + 2
    q = rng.standard_normal((rows, 4, 128))
    q[0, 0] = 0
    q[0, 1, 5] = np.nan
    q[1, 2, 0] = np.inf
    q[1, 3, 127] = -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        got, _ = attention_case(8, dtype, 4, 4, 128, 32, [100, 150], news, q=q)
    assert np.isnan(got[0, 1]).all() and not np.isnan(got[0, 0]).any() and np.isnan(got[1, 2:4]).all()
    for size, scale in ((1e-30, 1e29), (1e30, 1e-31)):
        attention_case(9, dtype, 4, 4, 128, 32, [100, 150], news, q_size=size, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 27, 2.0 ** 63, -2.0 ** 27, -2.0 ** 45, -2.0 ** 105])
@pytest.mark.parametrize("bound", [150, 2000])
def test_attention_scores_beyond_their_rounding(dtype, size, bound):
    """Scores so large that a unit of their float32 rounding passes the exponential's: the token of the largest score
    has all of the weight. Its weight is a power of two, so the output is its value, off by the reciprocals of the
    scale and of the sum, their product's sums and the last product (2^-23 and three times 2^-24: below 2^-21), and
    by bf16's 2^-8. Bound 150: rows in tiles of 16; 2000: of 256."""
    import torch
    kq = _kq()
    rng = np.random.default_rng(31)
    n, heads = 150, 4
    table, pages = tables(rng, [n], 16)
    cache = filled(rng, pages, 16, 1, 128)
    order = rng.permutation(n)                 # a score's size: 64 (2 + order) times the query's entry
    for t in range(n):
        at = cache.k[table[0][t // 16], 0, t % 16]
        at[:64] = 1 + order[t] // 2
        at[64:] = 1 + (order[t] + 1) // 2
    cache.k_scale[:] = 1.0
    q = _dev(np.full((max(bound, n), heads, 128), size), dtype)
    out = torch.zeros_like(q)
    kq.cache_attention(upload(cache), batch_of(table, [n], [0, n], bound), q, out, scale=0.5)
    got = out[:n].float().cpu().numpy().astype(np.float64)
    for i in range(n):
        t = max(range(i + 1), key=lambda x: order[x] * np.sign(size))
        page, slot = table[0][t // 16], t % 16
        want = cache.v[page, 0, slot // 16, :, slot % 16].astype(np.float64) * np.float64(cache.v_scale[page, 0])
        tol = np.abs(want) * (2.0 ** -21 + (2.0 ** -8 if dtype == "bf16" else 0.0))
        assert (np.abs(got[i] - want) <= tol).all(), (i, t)


def test_calls_with_nothing_to_do():
    """No rows, or no sequences: empty tensors pass through the binding and nothing is written."""
    import torch
    kq = _kq()
    dev = kq.KVCache.allocate(4, 16, 2, 64, DEV)
    before = [t.clone() for t in (dev.k, dev.v, dev.k_scale, dev.v_scale)]
    none = kq.CacheBatch(torch.zeros((0, 3), dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV),
                         torch.zeros(1, dtype=torch.int32, device=DEV), 5)
    for rows, batch in ((0, batch_of([[0, 1]], [7], [0, 0])), (0, none), (3, none)):
        q, kv = torch.ones((rows, 4, 64), device=DEV), torch.ones((rows, 2, 64), device=DEV)
        out, back = torch.full_like(q, 9.0), torch.full_like(kv, 9.0)
        kq.cache_append(dev, batch, q, kv, kv, out)
        kq.cache_append(dev, batch, None, kv, kv)
        kq.cache_attention(dev, batch, q, out)
        kq.cache_read(dev, batch, back, None)
        assert bool((out == 9.0).all()) and bool((back == 9.0).all())
    assert all(torch.equal(a, b) for a, b in zip(before, (dev.k, dev.v, dev.k_scale, dev.v_scale)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [[1], [3], [150]])
def test_attention_sees_no_poisoned_block_it_must_not(dtype, news):
    """A NaN scale reaches the rows that see its block and no others, also where the block shares a tile with what
    they see; a page that does not exist likewise, and is told."""
    kq = _kq()
    rng = np.random.default_rng(12)
    for where in (0, 7, 18):
        table, pages = tables(rng, [300], 16)
        cache = filled(rng, pages, 16, 2, 128)
        cache.v_scale[table[0][where], 1] = np.nan
        cache.k_scale[table[0][where], 0] = np.nan
        got, info = attention_case(13, dtype, 4, 2, 128, 16, [300], news, cache=cache, table=table)
        assert info == 0
        got, info = attention_case(13, dtype, 4, 2, 128, 16, [300], news, cache=cache, table=table, window=40)
        assert info == 0
        table[0][where] = pages + 3
        # the last row's window of 40 begins in block 16; the first row's, 300 - news + 1 - 40
        got, info = attention_case(13, dtype, 4, 2, 128, 16, [300], news, cache=cache, table=table)
        assert info == kq.KQ_INFO_PAGE
    # rows before the poisoned block of the same call
    table, pages = tables(rng, [160], 16)
    cache = filled(rng, pages, 16, 1, 64)
    cache.v_scale[table[0][9], 0] = np.nan
    got, _ = attention_case(14, dtype, 4, 1, 64, 16, [160], [150], cache=cache, table=table)
    assert not np.isnan(got[:134]).any() and np.isnan(got[134:150]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_many_sequences(dtype):
    """More sequences than are ordered by length (64), and exactly that many."""
    rng = np.random.default_rng(21)
    for n in (64, 70):
        lens = [int(x) for x in rng.integers(0, 90, n)]
        news = [int(rng.integers(0, x + 1)) for x in lens]
        attention_case(22, dtype, 4, 1, 64, 16, lens, news)


def test_bounds_far_above_the_rows():
    """max_q is a bound: one far above the rows asks for no more work or memory than the rows."""
    import torch
    kq = _kq()
    rng = np.random.default_rng(23)
    lens, q_start, page = [300, 20], [0, 5, 6], 32
    table, pages = tables(rng, lens, page)
    want = filled(rng, pages, page, 2, 64)
    dev = upload(want)
    b = batch_of(table, lens, q_start, 2 ** 31 - 1)
    x = rng.standard_normal((6, 8, 64)).astype(np.float32)
    xd, q, out = to_dev(x), torch.empty((6, 4, 64), device=DEV), torch.empty((6, 4, 64), device=DEV)
    k, v = (torch.empty((6, 2, 64), device=DEV) for _ in range(2))
    info = torch.zeros(1, dtype=torch.int32, device=DEV)
    kq.cache_append(dev, b, xd[:, :4], xd[:, 4:6], xd[:, 6:], q, info=info)
    ws = kq.cache_attention_workspace(dev, b, q)
    assert ws.numel() <= 64 * 2 ** 20
    kq.cache_attention(dev, b, q, out, ws=ws, window=2 ** 31 - 1, info=info)
    kq.cache_read(dev, b, k, v, info=info)
    x64 = x.astype(np.float64)
    kvcache.append(want, table, lens, q_start, x64[:, :4], x64[:, 4:6], x64[:, 6:])
    check_cache(dev, want)
    check_attention(host(out), want, table, lens, q_start, x[:, :4], 0.125, 0, "f32")
    wk = np.concatenate([kvcache.tokens(want, table[i], lens[i] - n, lens[i])[0] for i, n in enumerate((5, 1))])
    np.testing.assert_array_equal(host(k), wk.astype(np.float32))
    assert int(info.item()) == 0


def test_attention_wrong_entries_are_told():
    import torch
    kq = _kq()
    rng = np.random.default_rng(15)
    cache = filled(rng, 8, 16, 1, 64)
    dev = upload(cache)
    q20 = to_dev(rng.standard_normal((20, 2, 64)).astype(np.float32))

    def run(table, lens, q_start, max_q=20):
        q = q20
        if max_q > 20:                           # q_start's end past these rows is not past the call's
            q = torch.cat((q20, torch.zeros((max_q - 20, 2, 64), device=DEV)))
            q_start = [max_q + 1 if x == 21 else x for x in q_start]
        out, info = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device=DEV)
        kq.cache_attention(dev, batch_of(table, lens, q_start, max_q), q, out, info=info)
        return host(out), int(info.item())

    table = [[0, 1, 2, 3], [4, 5, 6, 7]]
    for bound in (20, 9000):                     # the single tokens' kernel and the prompts'
        good, info = run(table, [64, 40], [0, 10, 20], bound)
        assert info == 0
        for lens in ([64, -1], [64, 65], [2 ** 31 - 1, 40]):
            out, info = run(table, lens, [0, 10, 20], bound)
            assert info == kq.KQ_INFO_LENGTH
            if lens[1] == -1:
                assert not out[10:20].any()
            np.testing.assert_array_equal(out[:10], good[:10])  # 2^31 - 1 counts as the table's 64
        for q_start in ([0, 10, 21], [-1, 10, 20], [0, 12, 10]):
            _, info = run(table, [64, 40], q_start, bound)
            assert info == kq.KQ_INFO_ROWS
    out, info = run(table, [64, 40], [0, 10, 20], max_q=4)
    assert info == kq.KQ_INFO_ROWS


def test_attention_offsets_past_32_bits():
    """Pages whose codes begin past 2^31 and 2^32 bytes."""
    import torch
    kq = _kq()
    page, kvh, dim = 128, 8, 128
    pages = (2 ** 32) // (page * kvh * dim) + 40
    dev = kq.KVCache.allocate(pages, page, kvh, dim, DEV)
    rng = np.random.default_rng(16)
    small = filled(rng, 5, page, kvh, dim)
    far = [pages - 1, pages // 2 + 7, 3, pages - 20, pages // 2 - 1]
    at = torch.tensor(far, device=DEV)
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(dev, name)[at] = to_dev(getattr(small, name))
    for new, bound in ((1, None), (40, None), (40, 8192)):
        q = rng.standard_normal((new if bound is None else bound, 16, dim)).astype(np.float32)
        out = torch.empty(q.shape, device=DEV)
        kq.cache_attention(dev, batch_of([far], [600], [0, new], bound), to_dev(q), out)
        check_attention(host(out), small, [[0, 1, 2, 3, 4]], [600], [0, new], q, dim ** -0.5, 0, "f32")
    k, v = torch.empty((600, kvh, dim), device=DEV), torch.empty((600, kvh, dim), device=DEV)
    kq.cache_read(dev, batch_of([far], [600], [0, 600]), k, v)
    wk, wv = kvcache.tokens(small, [0, 1, 2, 3, 4], 0, 600)
    np.testing.assert_array_equal(host(k), wk.astype(np.float32))
    np.testing.assert_array_equal(host(v), wv.astype(np.float32))
    x = rng.standard_normal((100, 2 * kvh, dim)).astype(np.float32)
    xd = to_dev(x)
    kq.cache_append(dev, batch_of([far], [620], [0, 100]), None, xd[:, :kvh], xd[:, kvh:])
    kvcache.append(small, [[0, 1, 2, 3, 4]], [620], [0, 100], None, x[:, :kvh].astype(np.float64), x[:, kvh:].astype(np.float64))
    for name in ("k", "v", "k_scale", "v_scale"):
        np.testing.assert_array_equal(host(getattr(dev, name)[at]), getattr(small, name))
    del dev
    torch.cuda.empty_cache()


def test_calls_repeat_bit_for_bit_and_on_other_streams():
    """Two calls on two streams at once, each with its own workspace, equal a third one on the default stream."""
    import torch
    kq = _kq()
    rng = np.random.default_rng(17)
    table, pages = tables(rng, [4000, 900], 32)
    dev = upload(filled(rng, pages, 32, 2, 128))
    for news in ([1, 1], [200, 40], [3000, 600]):
        q = to_dev(rng.standard_normal((sum(news), 8, 128)).astype(np.float32))
        b = batch_of(table, [4000, 900], np.concatenate(([0], np.cumsum(news))))
        first = torch.empty_like(q)
        kq.cache_attention(dev, b, q, first)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [torch.empty_like(q) for _ in range(2)]
        for _ in range(3):
            for s, o in zip(streams, outs):
                kq.cache_attention(dev, b, q, o, stream=s)
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, first)


def test_graph_replays_with_new_contents():
    """A captured append, attention and read follow lengths, tables and rows that change between replays; eager
    calls run in between, and a second graph with its own workspace shares the cache."""
    import torch
    kq = _kq()
    from post_quantization_04_amd import pipeline
    rng = np.random.default_rng(18)
    page, kvh, heads, dim, steps = 16, 2, 8, 128, 6
    lens = [30, 700]
    table, pages = tables(rng, [n + steps for n in lens], page)
    want = filled(rng, pages, page, kvh, dim)
    dev = upload(want)
    rope = pipeline.rope_table(1000, dim)
    b = batch_of(table, lens, [0, 1, 2])
    x = torch.zeros((2, heads + 2 * kvh, dim), device=DEV)
    q, out = torch.empty((2, heads, dim), device=DEV), torch.empty((2, heads, dim), device=DEV)
    kr, vr = torch.empty((2, kvh, dim), device=DEV), torch.empty((2, kvh, dim), device=DEV)
    rd = rope.to(DEV)

    def step(ws):
        kq.cache_append(dev, b, x[:, :heads], x[:, heads:heads + kvh], x[:, heads + kvh:], q, rope=rd)
        kq.cache_attention(dev, b, q, out, ws=ws)
        kq.cache_read(dev, b, kr, vr)

    graphs = []
    wss = [kq.cache_attention_workspace(dev, b, q) for _ in range(2)]
    state = [t.clone() for t in (dev.k, dev.v, dev.k_scale, dev.v_scale)]
    step(wss[0])
    for ws in wss:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(ws)
        graphs.append(g)
    for t, saved in zip((dev.k, dev.v, dev.k_scale, dev.v_scale), state):
        t.copy_(saved)
    for i in range(steps):
        lens = [n + 1 for n in lens]
        xi = rng.standard_normal((2, heads + 2 * kvh, dim)).astype(np.float32)
        x.copy_(to_dev(xi))
        b.seq_lens.copy_(to_dev(np.asarray(lens, np.int32)))
        graphs[i % 2].replay()
        got, gk, gv = host(out), host(kr), host(vr)
        x64 = xi.astype(np.float64)
        wq = kvcache.append(want, table, lens, [0, 1, 2], x64[:, :heads], x64[:, heads:heads + kvh], x64[:, heads + kvh:],
                            rope=rope.numpy())
        check_cache(dev, want, f"step {i}")
        check_attention(got, want, table, lens, [0, 1, 2], wq.astype(np.float32), dim ** -0.5, 0, "f32")
        for r in range(2):
            wk, wv = kvcache.tokens(want, table[r], lens[r] - 1, lens[r])
            np.testing.assert_array_equal(gk[r], wk[0].astype(np.float32))
            np.testing.assert_array_equal(gv[r], wv[0].astype(np.float32))
        eager = torch.empty_like(out)
        kq.cache_attention(dev, b, q, eager)
        assert torch.equal(eager, out)


# ---- together, as they are used -----------------------------------------------------------------------------------


@pytest.mark.parametrize("graph", [False, True, "stream"])
def test_attention_step_on_quantized_weights(graph):
    """A prompt through append and attention, then single tokens through pipeline.attention_step (packed q, k, v, o
    layers, cache, attention), eager, as one captured graph or on a stream of its own, against the oracle fed with the same steps.

    The oracle's own chain feeds each step: decode matvec (2e-5 of the norm, as its own tests hold), then the cache.
    A key or value entry off by 2e-5 of its row can take another code, one step of its block's scale; so the step is
    compared from the library's own q, k and v on: the cache's codes and the attention exactly as above, the o
    projection at the decode matvec's 2e-5."""
    import torch

    import kq_synth
    import oracle
    kq = _kq()
    from post_quantization_04_amd import pipeline
    rng = np.random.default_rng(20)
    d, heads, kvh, dim, page, bits, group, n0, steps = 256, 4, 2, 64, 16, 4, 64, 21, 4
    lens = [n0, 5]
    table, pages = tables(rng, [n + steps for n in lens], page)
    want = kvcache.Cache.zeros(pages, page, kvh, dim)
    dev = upload(want)
    rope = pipeline.rope_table(64, dim)
    qw, kw = ((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    # the prompt
    x = rng.standard_normal((sum(lens), heads + 2 * kvh, dim)).astype(np.float32)
    xd = to_dev(x)
    q, out = torch.empty((sum(lens), heads, dim), device=DEV), torch.empty((sum(lens), heads, dim), device=DEV)
    q_start = [0, lens[0], sum(lens)]
    b = batch_of(table, lens, q_start)
    kq.cache_append(dev, b, xd[:, :heads], xd[:, heads:heads + kvh], xd[:, heads + kvh:], q, q_norm=to_dev(qw),
                    k_norm=to_dev(kw), rope=rope.to(DEV))
    kq.cache_attention(dev, b, q, out)
    x64 = x.astype(np.float64)
    kvcache.append(want, table, lens, q_start, x64[:, :heads], x64[:, heads:heads + kvh], x64[:, heads + kvh:], q_norm=qw,
                   k_norm=kw, rope=rope.numpy())
    check_cache(dev, want, "prompt")
    check_attention(host(out), want, table, lens, q_start, host(q), dim ** -0.5, 0, "f32")
    # the layers
    ri, s_x = kq_synth.rot_spec(31, "in", d), rng.uniform(0.3, 3.0, d)
    rio, s_xo = kq_synth.rot_spec(31, "oin", heads * dim), rng.uniform(0.3, 3.0, heads * dim)
    dri, drio = pipeline.upload_rot(ri.signs, ri.q, DEV), pipeline.upload_rot(rio.signs, rio.q, DEV)
    layers, host_layers, keep = [], [], []
    for name, dout, din in (("q", heads * dim, d), ("k", kvh * dim, d), ("v", kvh * dim, d), ("o", d, heads * dim)):
        codes = rng.integers(0, 1 << bits, size=(dout, din), dtype=np.uint8)
        scales = rng.uniform(0.005, 0.02, size=(dout, din // group)).astype(np.float32)
        zeros = rng.integers(0, 1 << bits, size=(dout, din // group), dtype=np.uint8)
        s_g, ro = rng.uniform(0.3, 3.0, dout), kq_synth.rot_spec(31, name, dout)
        packed = torch.zeros((dout, din * oracle.container_bits(bits) // 32), dtype=torch.int32, device=DEV)
        kq.pack_codes(to_dev(codes), bits, packed)
        keep.append(pipeline.upload_rot(ro.signs, ro.q, DEV))
        layers.append((packed, to_dev(scales), to_dev(zeros), to_dev(s_g), keep[-1].rot, torch.empty((2, dout), device=DEV)))
        host_layers.append((codes, scales, zeros, s_g, ro))
    step = kq.CacheBatch(to_dev(np.asarray(table, np.int32)), to_dev(np.asarray(lens, np.int32)),
                         to_dev(np.array([0, 1, 2], np.int32)), 1)
    xin = torch.zeros((2, d), device=DEV)
    ws = pipeline.attention_step_workspace(xin, layers[:3], layers[3], dev, step, heads)
    s_xd, s_xod, qwd, kwd, rd = to_dev(s_x), to_dev(s_xo), to_dev(qw), to_dev(kw), rope.to(DEV)

    def run(**kw):
        kw = kw or dict(ws=ws)
        return pipeline.attention_step(xin, layers[:3], layers[3], dev, step, heads, bits=bits, group=group, s_x=s_xd,
                                       rot_in=dri.rot, o_s_x=s_xod, o_rot_in=drio.rot, q_norm=qwd, k_norm=kwd, rope=rd, **kw)

    g = None
    if graph is True:
        saved = [t.clone() for t in (dev.k, dev.v, dev.k_scale, dev.v_scale)]
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        for t, s in zip((dev.k, dev.v, dev.k_scale, dev.v_scale), saved):
            t.copy_(s)
    for i in range(steps):
        lens = [n + 1 for n in lens]
        xi = rng.standard_normal((2, d)).astype(np.float32)
        xin.copy_(to_dev(xi))
        step.seq_lens.copy_(to_dev(np.asarray(lens, np.int32)))
        # the library's own q, k, v of this step (attention_step replaces q by its rotation)
        ref = [torch.empty_like(layer[5]) for layer in layers[:3]]
        kq.decode_matvec_group([(*layer[:5], r) for layer, r in zip(layers[:3], ref)], bits, group, s_xd, dri.rot, xin)
        for r, (codes, scales, zeros, s_g, ro) in zip(ref, host_layers):
            w = oracle.decode_matvec(codes, scales, zeros, group, s_x, s_g, ri, ro, xi)
            assert np.linalg.norm(host(r) - w) <= 2e-5 * np.linalg.norm(w)
        y = layers[3][5]
        if g is not None:
            g.replay()
        elif graph:
            torch.cuda.synchronize()
            first = run(stream=torch.cuda.Stream())                # buffers of its own
            torch.cuda.synchronize()
            first = first.clone()
            torch.cuda.synchronize()
            y = run(stream=torch.cuda.Stream(), ws=ws)             # the same token in the same place: the same cache
            torch.cuda.synchronize()
            assert torch.equal(first, y)
        else:
            y = run()
        qkv = [host(r).astype(np.float64).reshape(2, -1, dim) for r in ref]
        wq = kvcache.append(want, table, lens, [0, 1, 2], *qkv, q_norm=qw, k_norm=kw, rope=rope.numpy())
        check_cache(dev, want, f"step {i}")
        check_q(host(layers[0][5]).reshape(2, heads, dim), wq, "f32")
        attn = host(ws.attn)
        check_attention(attn.reshape(2, heads, dim), want, table, lens, [0, 1, 2], wq.astype(np.float32), dim ** -0.5, 0, "f32")
        codes, scales, zeros, s_g, ro = host_layers[3]
        w = oracle.decode_matvec(codes, scales, zeros, group, s_xo, s_g, rio, ro, attn)
        assert np.linalg.norm(host(y) - w) <= 2e-5 * np.linalg.norm(w)
