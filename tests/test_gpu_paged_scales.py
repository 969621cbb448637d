"""Scale bytes over their whole range, as a caller may fill them: 0 to 254 are
powers of two, 255 makes a row NaN."""
import pytest
import torch

import tests.pagedref as ref
from tests.test_gpu_paged import E4M3, E5M2, batch_of, filled, gen, on_gpu, sz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("D", [64, 128])
def test_every_scale_of_every_value_reads_back(dtype, D):
    """All 256 bytes with all 256 codes, K and V: the 64-bit value rounded once."""
    P, per = 16, 256 // D                                      # rows that hold every code
    rows = 256 * per
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(per, D)
    data = codes.repeat(256, 1).view(rows // P, 1, 1, P, D).repeat(1, 2, 1, 1, 1)
    scales = torch.arange(rows).div(per, rounding_mode="floor").to(torch.uint8).view(rows // P, 1, 1, P).repeat(1, 2, 1, 1)
    data = data.view(ref.ELEMENT[dtype])
    table = torch.arange(rows // P, dtype=torch.int32).view(1, -1)
    batch = batch_of(table, torch.tensor([rows], dtype=torch.int32), torch.tensor([0, rows], dtype=torch.int32), rows)
    k, v = sz().cache_read(on_gpu(dtype, data, scales), batch)
    want = ref.dequantise(data, scales)[:, 0, 0].reshape(rows, D).to(torch.bfloat16)
    want[255 * per:] = float("nan")
    for got in (k[:, 0].cpu(), v[:, 0].cpu()):
        same = (got.view(torch.int16) == want.view(torch.int16)) | (got.isnan() & want.isnan())
        assert bool(same.all()), (~same).nonzero()[:5].tolist()


@pytest.mark.parametrize("dtype,D", [(E5M2, 128), (E4M3, 64)])
@pytest.mark.parametrize("new", [1, 6, 60])
@pytest.mark.parametrize("byte", [0, 1, 255])
def test_attention_with_scales_at_the_ends(dtype, D, new, byte):
    """A row of K and V with such a byte, seen by every token, and another
    behind the sequence's end, seen by none."""
    H, G, P, n = 2, 4, 16, 330
    table, kv, starts, T, pages = ref.layout([n], [new], P, seed=3)
    data, scales = filled(dtype, pages, H, P, D, 4)
    for p in (100, n):
        scales[int(table[0, p // P]), :, :, p % P] = byte
    q = torch.randn(T, H * G, D, generator=gen(1)).to(torch.bfloat16)
    out, lse = sz().paged_attention(q.cuda(), on_gpu(dtype, data, scales),
                                    batch_of(table, kv, starts, T, max_new=new, max_kv=n), lse=True)
    if byte == 255:
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
    else:
        want, want_l, tol, tol_l = ref.attention(q, data, scales, table, kv, starts, P, D ** -0.5, 0)
        assert not ref.close(out, want, tol)
        assert not ref.close(lse, want_l, tol_l)
    # a window that hides the first row leaves neither
    if new < 60:
        out, lse = sz().paged_attention(q.cuda(), on_gpu(dtype, data, scales),
                                        batch_of(table, kv, starts, T, max_new=new, max_kv=n), window=200, lse=True)
        want, want_l, tol, tol_l = ref.attention(q, data, scales, table, kv, starts, P, D ** -0.5, 200)
        assert not ref.close(out, want, tol)
        assert not ref.close(lse, want_l, tol_l)
