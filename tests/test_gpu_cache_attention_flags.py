"""A bad page that one warp of a block meets: its sequence's output is NaN and the plan reports it, whatever the block's
shared memory held before."""
import pytest
import torch

from fp8_implicit_gemm_gb300 import capi, q8
from _attention_common import CODE_ARG, fill_cache, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codes", ["i4", "i8"])
@pytest.mark.parametrize("seqs", [1, 32, 33])
def test_a_bad_page_of_any_warp_is_reported(codes, seqs):
    heads, kv, dim, width = 8, 1, 128, 9
    cache = q8.CacheQ8.empty(seqs * width, 16, kv, dim, CODE_ARG[codes])
    fill_cache(cache, codes, 1)
    table = torch.arange(seqs * width, dtype=torch.int32, device="cuda").view(seqs, width)
    lengths = torch.full((seqs,), 16 * width - 3, dtype=torch.int32, device="cuda")
    q = randn(seqs, heads, dim, dtype=torch.bfloat16, seed=2)
    attend = q8.CacheAttention(cache, heads, max_seqs=seqs)
    want = attend(q, table, lengths, torch.empty_like(q)).clone()
    assert attend.check() == capi.CONV3D_OK
    # a kernel that leaves the blocks' shared memory full of values
    codes8 = torch.full((4096, 1024), 0x77, dtype=torch.int8, device="cuda")
    ones = torch.ones(4096, device="cuda")
    product = q8.LinearQ8(codes8, ones, max_rows=4096)
    spare = torch.empty(4096, 4096, dtype=torch.bfloat16, device="cuda")
    for place in range(width):
        for bad in (seqs * width, -1):
            b = place % seqs
            keep = int(table[b, place])
            table[b, place] = bad
            product(codes8, ones, spare)
            o = attend(q, table, lengths, torch.full_like(q, 7.0))
            assert attend.check() == capi.CONV3D_EDEVICE
            assert bool(torch.isnan(o[b]).all())
            others = [i for i in range(seqs) if i != b]
            assert torch.equal(o[others], want[others])
            table[b, place] = keep
            product(codes8, ones, spare)
            assert torch.equal(attend(q, table, lengths, torch.full_like(q, 7.0)), want)
            assert attend.check() == capi.CONV3D_OK


def test_a_check_does_not_clear_what_the_next_run_reports():
    """Runs on a stream that the default one does not order, each with a bad page, each reported."""
    cache = q8.CacheQ8.empty(4, 16, 1, 64)
    table = torch.full((1, 1), 9, dtype=torch.int32, device="cuda")
    length, q = torch.ones(1, dtype=torch.int32, device="cuda"), randn(1, 1, 64, dtype=torch.bfloat16, seed=1)
    attend, o, s = q8.CacheAttention(cache, 1), torch.empty_like(q), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(300):
        attend(q, table, length, o, stream=s)
        assert attend.check() == capi.CONV3D_EDEVICE
    assert attend.check() == capi.CONV3D_OK
