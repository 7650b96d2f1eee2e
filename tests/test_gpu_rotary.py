"""pa_rotary against the oracle: types, layouts, parts of the head, positions,
strides, special values, the transposed rotation."""

import numpy as np
import pytest
import torch

import pagedattention_decode_attention_gb300 as pa
from oracle import rotary as orot
from pagedattention_decode_attention_gb300 import workloads as wl
from tests.gpu_helpers import TORCH_DTYPES, to_f32_numpy
from tests.rotary_helpers import LONG, angle_error, projection, rotary_of, rotation_bound, same_bits
from tests.window_helpers import HALF_STEP, assert_within

pytestmark = pytest.mark.gpu

# near, far, the ends of 32 bits, behind zero
POSITIONS = [0, 1, 2, 7, 63, 64, 100, 4095, 65537, 131071, 1000003, 2 ** 24 + 1, 2 ** 31 - 1, -1, -100, -2 ** 31]


def check(got, x, positions, w, rot, dtype):
    ref, size = orot.rotate(to_f32_numpy(x), positions, w, rot.interleaved, rot.magnitude)
    assert_within(got, ref, rotation_bound(ref, size, positions, w, dtype))
    # what is not rotated keeps its bits
    assert same_bits(got[..., rot.rotary_dim:], x[..., rot.rotary_dim:])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("part", ["all", "half", "sixteen", "but sixteen"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads", [(32, 8), (5, 1), (3, 3)], ids=str)
def test_matches_oracle(gpu, dtype, head_dim, part, interleaved, heads):
    rdim = {"all": head_dim, "half": head_dim // 2, "sixteen": 16, "but sixteen": head_dim - 16}[part]
    rot, w = rotary_of(pa, head_dim, gpu, rdim, interleaved, 1.0 if interleaved else 1.25)
    n = len(POSITIONS)
    q, k, _ = projection(n, *heads, head_dim, dtype, 11 + rdim, gpu, pad=16)
    pos = torch.tensor(POSITIONS, dtype=torch.int64).to(torch.int32).to(gpu)
    qo, ko = pa.rotary(q, k, pos, rot)
    pa.check_status()
    check(qo, q, POSITIONS, w, rot, dtype)
    check(ko, k, POSITIONS, w, rot, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=2.5), LONG],
                         ids=lambda c: c["scaling"])
def test_long_contexts(gpu, dtype, scaling):
    rot, w = rotary_of(pa, 128, gpu, magnitude=0.1 * np.log(scaling["factor"]) + 1, **scaling)
    positions = list(range(30000, 30050)) + [4096, 8191]
    q, k, _ = projection(len(positions), 4, 2, 128, dtype, 5, gpu)
    qo, ko = pa.rotary(q, k, torch.tensor(positions, dtype=torch.int32, device=gpu), rot)
    check(qo, q, positions, w, rot, dtype)
    check(ko, k, positions, w, rot, dtype)


@pytest.mark.parametrize("n", [0, 1, 2, 3, 31, 515])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_lengths(gpu, n, head_dim):
    rot, w = rotary_of(pa, head_dim, gpu)
    q, k, _ = projection(n, 7, 3, head_dim, "bf16", 3 + n, gpu)
    pos = torch.arange(n, dtype=torch.int32, device=gpu) * 3
    qo, ko = pa.rotary(q, k, pos, rot)
    pa.check_status()
    assert qo.shape == q.shape and ko.shape == k.shape and qo.is_contiguous()
    if n:
        check(qo, q, (np.arange(n) * 3).tolist(), w, rot, "bf16")
        check(ko, k, (np.arange(n) * 3).tolist(), w, rot, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_alone_and_prepared(gpu, dtype, interleaved):
    rot, _ = rotary_of(pa, 128, gpu, 96, interleaved)
    n = 77
    x = wl.normal((n, 12 * 128 + 32), TORCH_DTYPES[dtype], 9, gpu)
    whole = x.clone()
    q, k = x[:, : 8 * 128].unflatten(1, (8, 128)), x[:, 8 * 128: 10 * 128].unflatten(1, (2, 128))
    pos = torch.randint(0, 9999, (n,), dtype=torch.int32, device=gpu)
    qo, ko = pa.rotary(q, k, pos, rot)
    only_q, none = pa.rotary(q, None, pos, rot)
    none2, only_k = pa.rotary(None, k, pos, rot)
    assert none is None and none2 is None
    assert same_bits(only_q, qo) and same_bits(only_k, ko)
    again_q, again_k = torch.empty_like(qo), torch.empty_like(ko)
    op = pa.prepare_rotary(q, k, pos, rot, again_q, again_k)
    op()
    assert same_bits(again_q, qo) and same_bits(again_k, ko)
    assert torch.equal(x, whole)                    # the inputs stand
    pa.rotary(q, k, pos, rot, q_out=q, k_out=k)     # in place, in the middle of wider rows
    assert same_bits(q, qo) and same_bits(k, ko)
    assert torch.equal(x[:, 10 * 128:], whole[:, 10 * 128:])
    pa.check_status()


def test_rows_that_repeat(gpu):
    """A stride of zero: one row at many positions."""
    rot, _ = rotary_of(pa, 64, gpu)
    one = wl.normal((1, 4, 64), torch.float16, 3, gpu)
    pos = torch.arange(50, dtype=torch.int32, device=gpu)
    a, b = pa.rotary(one.expand(50, 4, 64), one.expand(50, 4, 64)[:, :2], pos, rot)
    c, d = pa.rotary(one.repeat(50, 1, 1), one.repeat(50, 1, 1)[:, :2], pos, rot)
    assert same_bits(a, c) and same_bits(b, d)
    with pytest.raises(ValueError, match="overlap"):
        pa.rotary(c, None, pos, rot, q_out=torch.empty((1, 4, 64), dtype=torch.float16, device=gpu).expand(50, 4, 64))


def test_what_the_binding_refuses(gpu):
    rot, _ = rotary_of(pa, 64, gpu)
    x = torch.zeros(4, 8, 64, dtype=torch.bfloat16, device=gpu)
    pos = torch.zeros(4, dtype=torch.int32, device=gpu)
    bad = [lambda: pa.rotary(x.transpose(0, 1), None, pos, rot),                    # heads apart
           lambda: pa.rotary(x[..., ::2], None, pos, rot),
           lambda: pa.rotary(x, x[:3], pos, rot),
           lambda: pa.rotary(x, x.float(), pos, rot),
           lambda: pa.rotary(x, None, pos.long(), rot),
           lambda: pa.rotary(x, None, pos[:3], rot),
           lambda: pa.rotary(x, None, pos.cpu(), rot),
           lambda: pa.rotary(x, None, pos, pa.Rotary(128, gpu)),
           lambda: pa.rotary(x, None, pos, pa.Rotary(64, "cpu")),
           lambda: pa.rotary(x, None, pos, rot, k_out=x),
           lambda: pa.rotary(x, None, pos, rot, q_out=x[:, :4])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros(4 * 516, dtype=torch.bfloat16, device=gpu).view(4, 516)[:, :512].unflatten(1, (8, 64))
    with pytest.raises(pa.PagedAttnError):          # rows 8 bytes off a vector
        pa.rotary(odd, None, pos, rot)
    with pytest.raises(TypeError):
        pa.rotary(x.to(torch.float8_e4m3fn), None, pos, rot)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_special_values(gpu, dtype, interleaved):
    """Infinities and NaN stay with their pair; the type's largest and smallest
    are rounded once (f16's largest may pass its range, to infinity)."""
    rot, w = rotary_of(pa, 64, gpu, 64, interleaved)
    dt = TORCH_DTYPES[dtype]
    x = wl.normal((6, 3, 64), dt, 3, gpu)
    first, second = orot.pair_columns(64, interleaved)
    x[0, 0, int(first[3])] = float("inf")
    x[1, 1, int(second[5])] = float("nan")
    x[2, 2] = torch.finfo(dt).max
    x[3, 0] = torch.finfo(dt).smallest_normal
    x[4] = 0.0
    positions = [0, 5, 40, 41, 42, 1]
    got, _ = pa.rotary(x, None, torch.tensor(positions, dtype=torch.int32, device=gpu), rot)
    ref, size = orot.rotate(to_f32_numpy(x), positions, w, interleaved)
    out = to_f32_numpy(got).astype(np.float64)
    odd = np.zeros(out.shape, dtype=bool)
    odd[0, 0, [first[3], second[3]]] = True
    odd[1, 1, [first[5], second[5]]] = True
    # position 0 of (inf, b): inf * 1 - b * 0, and b * 1 + inf * 0
    assert out[0, 0, first[3]] == np.inf and np.isnan(out[0, 0, second[3]])
    assert np.isnan(out[1, 1, [first[5], second[5]]]).all()
    largest = float(torch.finfo(dt).max)
    limit = rotation_bound(np.where(odd, 0, ref), np.where(odd, 0, size), positions, w, dtype)
    over = np.abs(ref) > largest
    assert (~np.isfinite(out[over]) | (np.abs(out[over]) >= largest * (1 - HALF_STEP[dtype]))).all()
    fine = ~odd & (np.abs(ref) <= largest * (1 - 2 * HALF_STEP[dtype]))
    assert fine.sum() > out.size // 2
    assert (np.abs(out[fine] - ref[fine]) <= limit[fine]).all()
    assert (out[4] == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rdim", [32, 128])
def test_transposed_is_the_gradient(gpu, interleaved, rdim):
    """f(x) = sum g * rotary(x): the gradient by the formula (the transposed
    matrix, built column by column from the oracle), and by differences."""
    rot, w = rotary_of(pa, 128, gpu, rdim, interleaved, 1.3)
    positions = [0, 3, 1000, 70000]
    pos = torch.tensor(positions, dtype=torch.int32, device=gpu)
    g = wl.normal((4, 2, 128), torch.float32, 7, gpu)
    grad, grad_k = pa.rotary(g, g, pos, rot.transposed())
    assert same_bits(grad, grad_k)
    g64 = to_f32_numpy(g).astype(np.float64)
    eye = np.eye(128)[:, None]
    _, size = orot.rotate(g64, positions, w, interleaved, 1.3)
    limit = rotation_bound(g64, size, positions, w, "f32")
    got = to_f32_numpy(grad).astype(np.float64)
    for t, p in enumerate(positions):
        matrix = orot.rotate(eye, [p] * 128, w, interleaved, 1.3)[0][:, 0].T      # y = matrix x
        assert (np.abs(got[t] - g64[t] @ matrix) <= limit[t]).all()
    # differences: a linear map's are its slopes.  x + 1 and x - 1 are rounded,
    # then rotated: 8 + 2 half steps of the pairs' sums, each weighed by |g|
    x = wl.normal((4, 2, 128), torch.float32, 8, gpu)
    around = np.abs(to_f32_numpy(x).astype(np.float64)) + 1
    _, size = orot.rotate(around, positions, w, interleaved, 1.3)
    room = (np.abs(g64) * (10 * size + 2 * around)).sum(-1) * HALF_STEP["f32"]
    room = room + (np.abs(g64) * size).sum(-1) * angle_error(positions, w)[:, :, 0]
    for column in (0, 1, 17, rdim // 2, rdim - 1, 127):
        step = torch.zeros_like(x)
        step[..., column] = 1.0
        up, down = pa.rotary(x + step, None, pos, rot)[0], pa.rotary(x - step, None, pos, rot)[0]
        slope = ((up.double() - down.double()) * g.double()).sum(-1).cpu().numpy() / 2
        assert (np.abs(slope - got[..., column]) <= room + limit[..., column]).all()


def test_there_and_back(gpu):
    """The transposed rotation undoes one of magnitude 1, at far positions too."""
    rot, _ = rotary_of(pa, 64, gpu)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (999,), dtype=torch.int64, device=gpu).to(torch.int32)
    x = wl.normal((999, 4, 64), torch.float32, 8, gpu)
    there, _ = pa.rotary(x, None, pos, rot)
    back, _ = pa.rotary(there, None, pos, rot.transposed())
    # the first turn's error, at most 8 half steps of the pair's sum in either
    # column, turned back: 16; the second's, 8 of a sum at most sqrt 2 as large
    size = (x.abs() + x.roll(32, -1).abs())
    assert ((back - x).abs() <= 28 * HALF_STEP["f32"] * size).all()


def test_products_depend_on_the_distance(gpu):
    rot, _ = rotary_of(pa, 128, gpu, magnitude=1.0)
    q, k = (wl.normal((1, 1, 128), torch.float32, s, gpu) for s in (1, 2))
    starts = [0, 5, 100000, 2 ** 30]
    qs, ks = q.expand(4, 1, 128), k.expand(4, 1, 128)
    a, _ = pa.rotary(qs, None, torch.tensor([s + 77 for s in starts], dtype=torch.int32, device=gpu), rot)
    b, _ = pa.rotary(ks, None, torch.tensor(starts, dtype=torch.int32, device=gpu), rot)
    dots = (a.double() * b.double()).sum(-1)[:, 0]
    # every value is off by at most 8 half steps of its pair's sum, itself at
    # most sqrt 2 times the rotated pair's; both dots; the angles' difference is
    # exact
    a, b = a.double().abs(), b.double().abs()
    sa, sb = (2 ** 0.5 * (x + x.roll(64, -1)) for x in (a, b))
    room = 2 * 8 * HALF_STEP["f32"] * (sa * b + a * sb).sum(-1).max() * (1 + 2.0 ** -10)
    assert (dots - dots[0]).abs().max() <= room


def test_streams_and_graphs(gpu):
    """On another stream, and captured with eager calls in between; every
    replay gives what the eager call gives."""
    rot, _ = rotary_of(pa, 128, gpu, interleaved=True)
    q, k, _ = projection(300, 8, 2, 128, "bf16", 4, gpu)
    pos = torch.arange(300, dtype=torch.int32, device=gpu)
    want = pa.rotary(q, k, pos, rot)
    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream(gpu))
    got = pa.rotary(q, k, pos, rot, stream=side)
    torch.cuda.current_stream(gpu).wait_stream(side)
    assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
    out = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.rotary(q, k, pos, rot, *out)
    for shift in (0, 1000):
        pos += shift
        graph.replay()
        want = pa.rotary(q, k, pos, rot)
        assert same_bits(out[0], want[0]) and same_bits(out[1], want[1])
    pa.check_status()


def test_rows_past_32_bit_offsets(gpu):
    """Rows so far apart that their elements' numbers pass 32 bits."""
    rot, _ = rotary_of(pa, 64, gpu)
    stride, n = 1 << 22, 600                            # 2.5e9 elements
    wide = torch.zeros(n * stride, dtype=torch.bfloat16, device=gpu).view(n, stride)
    x = wl.normal((n, 2, 64), torch.bfloat16, 6, gpu)
    wide[:, :128] = x.flatten(1)
    pos = torch.arange(n, dtype=torch.int32, device=gpu)
    rows = wide[:, :128].unflatten(1, (2, 64))
    want, _ = pa.rotary(x, None, pos, rot)
    got, _ = pa.rotary(rows, None, pos, rot)
    assert same_bits(got, want)
    pa.rotary(rows, None, pos, rot, q_out=rows)
    assert same_bits(rows, want)
    assert float(wide[-1, 128:4096].float().abs().max()) == 0
