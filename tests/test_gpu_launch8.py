"""The 8-bit layer's calls on sizes that one launch cannot cover (HIP takes
fewer than 2^32 work items in a dimension): they are done in parts.  Narrow
rows, so that the memory fits; values are checked in the first rows, around the
parts' borders and in the last."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def room(gib):
    """Skips where the card has less memory than the test takes."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def test_adamw_of_many_elements():
    """33 tensors of 2^30 and more elements in one call, reading one gradient; borders of launches lie inside tensors."""
    sizes = [(1 << 30) + 24 * i + (i % 8) for i in range(33)]
    say(f"adamw on {sum(sizes)} elements")
    room(160)
    assert sum(sizes) > 1 << 35
    g = torch.ones(max(sizes), dtype=BF, device=DEV)
    g[1::2] = -1.0
    u8 = lambda n, v: torch.full((n,), v, dtype=torch.uint8, device=DEV)  # noqa: E731
    p = [torch.zeros(n, dtype=BF, device=DEV) for n in sizes]
    m, v = [u8(n, 0) for n in sizes], [u8(n, 0) for n in sizes]
    ms, vs = ([u8(-(-n // 128), 127) for n in sizes] for _ in range(2))
    t = ng.AdamWTensors(p, [g[:n] for n in sizes], m, v, ms, vs)
    ng.ngram_adamw(t, lr=1e-2, step=1)
    for i in range(33):
        # every element moved by lr against its gradient's sign, once, to within a bf16 step
        lo, hi = (p[i][0::2].min(), p[i][0::2].max()), (p[i][1::2].min(), p[i][1::2].max())
        assert all(abs(float(a) + 1e-2) <= 1e-4 for a in lo) and all(abs(float(a) - 1e-2) <= 1e-4 for a in hi), i
        assert int(v[i].min()) > 0 and int(vs[i].max()) < 127 and int(ms[i].max()) < 127, i
    # the random words go on where a tensor is cut: equal to the step on the tail alone with its place in the sequence
    i, cut = 31, 1 << 29
    assert sum(sizes[:i]) + cut < (1 << 35) - 2048 < sum(sizes[:i + 1])
    q, qm, qv = torch.zeros(sizes[i] - cut, dtype=BF, device=DEV), u8(sizes[i] - cut, 0), u8(sizes[i] - cut, 0)
    qs = [u8(-(-(sizes[i] - cut) // 128), 127) for _ in range(2)]
    place = sum(-(-n // 128) * 128 for n in sizes[:i]) + cut
    ng.ngram_adamw(ng.AdamWTensors([q], [g[cut:sizes[i]]], [qm], [qv], [qs[0]], [qs[1]], rng_offsets=[place]), lr=1e-2, step=1)
    assert torch.equal(q, p[i][cut:]) and torch.equal(qm, m[i][cut:]) and torch.equal(qv, v[i][cut:])


@pytest.mark.parametrize("listed", [True, False])
def test_adamw_rows_of_many_narrow_rows(listed):
    room_for, R, d = (1 << 28) + 333, (1 << 28) + 500, 8     # a group of 16 lanes a row
    say(f"adamw_rows, {room_for} rows of {d}")
    room(20)
    p = torch.zeros((R, d), dtype=BF, device=DEV)
    m, v = (torch.zeros((R, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.full((R, 1), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    rows = torch.arange(100, room_for + 100, dtype=torch.int32, device=DEV)
    g = torch.ones((room_for, d), dtype=BF, device=DEV)
    g[1::2] = -1.0
    count = room_for - 50 if listed else room_for
    n_rows = torch.tensor([count], device=DEV) if listed else None
    ng.ngram_adamw_rows(p, m, v, rows, g, n_rows, m_scale=ms, v_scale=vs, lr=1e-2, step=1)
    assert not bool(p[:100].any()) and not bool(p[100 + count:].any()) and not bool(v[100 + count:].any())
    hit = p[100:100 + count]
    assert float((hit[0::2].float() + 1e-2).abs().max()) <= 1e-4 and float((hit[1::2].float() - 1e-2).abs().max()) <= 1e-4
    # the random words go by the row: the same as the step on the last rows alone
    q, qm, qv = torch.zeros_like(p[:R]), torch.zeros_like(m), torch.zeros_like(v)
    qs = [torch.full((R, 1), 127, dtype=torch.uint8, device=DEV) for _ in range(2)]
    a, b = count - 1001, count
    ng.ngram_adamw_rows(q, qm, qv, rows[a:b], g[a:b], m_scale=qs[0], v_scale=qs[1], lr=1e-2, step=1)
    assert torch.equal(q[100 + a:100 + b], p[100 + a:100 + b]) and torch.equal(qv[100 + a:100 + b], v[100 + a:100 + b])


def test_norm_of_many_narrow_rows():
    n, d = (1 << 26) + 77, 8                            # 64 threads a row
    say(f"norm {n} x {d}")
    room(24)
    x = torch.randn((n, d), device=DEV).to(BF)
    gamma = torch.rand(d, device=DEV)
    s, y = torch.empty_like(x), torch.empty_like(x)
    res = torch.zeros_like(x)
    res[-1000:] = 1.0
    out = ng.ngram_add_norm(x, gamma, 1e-6, residual=res, sum_out=s, y_out=y, keep_r=True)
    assert torch.equal(s[:-1000], x[:-1000]) and torch.equal(s[-1000:], x[-1000:] + res[-1000:])
    for a, b in ((0, 5000), ((1 << 26) - 3000, n), ((1 << 25) - 3000, (1 << 25) + 3000)):
        few = ng.ngram_add_norm(s[a:b].contiguous(), gamma, 1e-6, keep_y=True, keep_r=True)
        assert torch.equal(out.r[a:b], few.r) and torch.equal(y[a:b], few.y)
        assert torch.equal(out.q.codes[a:b].view(torch.uint8), few.q.codes.view(torch.uint8))
        assert torch.equal(out.q.scales[a:b], few.q.scales)
    want = torch.rsqrt((s.float() ** 2).mean(dim=1) + 1e-6)
    assert torch.all((out.r - want).abs() <= 1e-5 * want)


def test_norm_of_many_wide_rows():
    n, d = (1 << 22) + 9, 8192                          # 16 wavefronts a row
    say(f"norm {n} x {d}")
    room(80)
    x = torch.zeros((n, d), dtype=BF, device=DEV)
    x.view(-1)[::4096] = 1.0
    r = torch.zeros(n, device=DEV)
    ng.ngram_add_norm(x, torch.ones(d, device=DEV), 1.0, quantise=False, r_out=r)
    at = torch.arange(n, device=DEV) * d
    ones = (at + d + 4095) // 4096 - (at + 4095) // 4096
    want = torch.rsqrt(ones / d + 1.0)
    assert torch.all((r - want).abs() <= 1e-6)


def test_product_of_few_rows_with_many():
    n, k = (1 << 26) + 136, 128                         # 64 threads an output column
    say(f"product 2 x {n} x {k}")
    room(16)
    codes = torch.full((n, k), 0x38, dtype=torch.uint8, device=DEV)          # 1
    codes[::3] = 0x40                                                        # 2
    for block_rows in (1, 128):
        rows = n if block_rows == 1 else -(-n // 128)
        scales = (127 + torch.arange(rows, device=DEV) % 3).to(torch.uint8)[:, None].repeat(1, 4)
        b = ng.Fp8(codes, scales, n, k, block_rows=block_rows)
        a = ng.Fp8(torch.full((2, k), 0x38, dtype=torch.uint8, device=DEV), torch.tensor([[127] * 4, [128] * 4], dtype=torch.uint8, device=DEV), 2, k)
        got = ng.ngram_project_fp8(a, b)
        i = torch.arange(n, device=DEV)
        want = 128.0 * torch.where(i % 3 == 0, 2.0, 1.0) * 2.0 ** ((i if block_rows == 1 else i // 128) % 3)
        assert torch.equal(got[0].float(), want) and torch.equal(got[1].float(), 2 * want)


def test_product_of_very_many_rows():
    m, n, k = 1 << 30, 8, 128                           # 2^23 tiles of 512 threads
    say(f"product {m} x {n} x {k}")
    room(170)
    a_codes = torch.full((m, k), 0x38, dtype=torch.uint8, device=DEV)
    b_codes = torch.full((n, k), 0x38, dtype=torch.uint8, device=DEV)
    one = lambda r: torch.full((-(-r // 128), 4), 127, dtype=torch.uint8, device=DEV)  # noqa: E731
    a_s, b_s = one(m), one(n)
    a_s[::2] = 128
    got = ng.ngram_project_fp8(ng.Fp8(a_codes, a_s, m, k, block_rows=128), ng.Fp8(b_codes, b_s, n, k, block_rows=128))
    got = got.view(-1, 2, 128, n)
    for part, want in ((got[:, 0], 256.0), (got[:, 1], 128.0)):
        lo, hi = torch.aminmax(part)
        assert float(lo) == want and float(hi) == want
