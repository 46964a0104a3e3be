"""What sv_sync says of bad calls on a cache: sequences without rows, far offsets, errors of two kinds at once."""
import pytest
import torch

import cache_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("count,bad", [(3, 1), (100, 0), (100, 99), (2000, 1234)])
@pytest.mark.parametrize("length", [-1, 33, 2 ** 31 - 1])
def test_lengths_of_sequences_without_rows(sv, read, count, bad, length):
    """Reported as sv_attention_cached reports them; the sequences with rows are served."""
    few = count > 1000  # rows of the first sequences alone: a warp checks more than 32
    have = [0 if few and i > 20 else 5 + i % 7 for i in range(count)]
    b = cache_ref.Batch(have, 16, 2, 64, prefix=20, seed=1, fill=0)
    b.stride = 2
    b.table = torch.nn.functional.pad(b.table, (0, 2 - b.table.shape[1]), value=-7)
    for i in range(count):
        for which in range(2 if have[i] else 0):
            b.pool.store(which, *b.places(i, 0, have[i]), torch.full((have[i], 2, 64), 0.25 * (i % 8 + which), device="cuda").half())
    n = [min(i % 3, have[i]) for i in range(count)]
    n[bad] = 0
    off = torch.tensor([0] + n).cumsum(0).to(torch.int32).cuda()
    total = sum(n)
    rows = torch.full((total, 128), 3.0, device="cuda", dtype=torch.float16)
    k, v = rows.clone(), rows.clone()
    call = sv.sv_cache_read if read else sv.sv_cache_write
    for spoiled in (False, True):
        if spoiled:
            b.lengths[bad] = length
        if read:
            k.copy_(rows), v.copy_(rows)
        call(b.cache(sv), b.batch(sv), k, v, off, total)
        if spoiled:
            with pytest.raises(sv.SvError) as e:
                sv.sv_sync()
            assert e.value.status == sv.SV_ERR_INVALID_ARG and "cache" in str(e.value)
        sv.sv_sync()
        for i in range(21 if few else count):
            row = int(off[i])
            for which, x in enumerate((k, v)):
                stored = b.pool.values(which, *b.places(i, have[i] - n[i], have[i]))
                assert torch.equal(stored.reshape(n[i], 128), x[row:row + n[i]].double())


@pytest.mark.parametrize("read", [False, True])
def test_offsets_of_the_last_sequences(sv, read):
    """Offsets that decrease far behind the rows of the call's first warp."""
    count = 1000
    b = cache_ref.Batch([9] * count, 16, 1, 64, seed=1, fill=0)
    b.fill(1)
    off = (torch.arange(count + 1) // 2).to(torch.int32).cuda()
    off[991:994] = torch.tensor([495, 494, 496], dtype=torch.int32)
    k, v = (torch.zeros(count // 2, 64, device="cuda", dtype=torch.float16) for _ in range(2))
    (sv.sv_cache_read if read else sv.sv_cache_write)(b.cache(sv), b.batch(sv), k, v, off, count // 2)
    with pytest.raises(sv.SvError) as e:
        sv.sv_sync()
    assert e.value.status == sv.SV_ERR_INVALID_ARG and "cache" in str(e.value)
    sv.sv_sync()


def test_errors_of_two_kinds(sv):
    """Bad documents and a bad cache before one sv_sync: it names both."""
    q = torch.zeros(4, 64, device="cuda", dtype=torch.float16)
    o = torch.empty_like(q)
    bad = torch.tensor([0, 3, 2, 4], dtype=torch.int32, device="cuda")
    b = cache_ref.Batch([4, 4, 4], 16, 1, 64, seed=1, fill=0)
    packed = lambda: sv.sv_attention_packed(q, q, q, o, bad, bad, 3, 4, 4, 1, 1, 64)
    write = lambda: sv.sv_cache_write(b.cache(sv), b.batch(sv), q, q, bad, 4)
    for calls, names in (((packed,), ("sv_attention_packed",)), ((write,), ("cache",)),
                         ((packed, write), ("sv_attention_packed", "cache"))):
        for call in calls:
            call()
        with pytest.raises(sv.SvError) as e:
            sv.sv_sync()
        assert e.value.status == sv.SV_ERR_INVALID_ARG
        for name in ("sv_attention_packed", "cache"):
            assert (name in str(e.value)) == (name in names)
        sv.sv_sync()
