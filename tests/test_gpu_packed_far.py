"""sv_attention_packed at positions behind 2^24, where a position is no F32 number any more."""
import pytest
import torch

import packed_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lq,hq,hk,d", [(1, 2, 2, 8), (3, 2, 1, 8), (20, 1, 1, 8), (1, 4, 1, 72)])
@pytest.mark.parametrize("softcap", [0.0, 4.0])
def test_distance_bias_far_into_a_document(sv, lq, hq, hk, d, softcap):
    """One document of 2^24 + 40,001 keys, scores that fall by a slope of 1 or more a key: only the last keys matter,
    and the reference takes those behind the 2,000th from the end (the others have weights below 2^-1000)."""
    n, near = 2 ** 24 + 40001, 2000
    gen = torch.Generator("cuda").manual_seed(d + lq)
    k = torch.randn(n, hk * d, generator=gen, device="cuda", dtype=torch.float16)
    v = torch.randn(n, hk * d, generator=gen, device="cuda", dtype=torch.float16)
    q = torch.randn(lq, hq * d, generator=gen, device="cuda", dtype=torch.float16)
    slopes = torch.linspace(1.0, 1.5, hq, device="cuda")
    o = torch.empty_like(q)
    ws = torch.zeros(sv.sv_attention_packed_workspace(1, lq, n, hq, hk, d), dtype=torch.uint8, device="cuda")
    for mask in (0, 1):
        opt = sv.sv_attention_options(softcap=softcap, mask=mask, slopes=slopes)
        for workspace in (ws, None):
            o.fill_(float("nan"))
            sv.sv_attention_packed(q, k, v, o, None, None, 1, lq, n, hq, hk, d, options=opt, workspace=workspace)
            sv.sv_sync()
            kn, vn = (x[n - near:].reshape(near, hk, d) for x in (k, v))
            ref, av, terms = packed_ref.document(q.view(lq, hq, d), kn, vn, mask, softcap=softcap, slopes=slopes)
            # (the bias of the keys that count is below 2^6, so F32 holds it to 2^-18; terms are those of all `near` keys)
            tol = packed_ref.bound(ref, av, terms.clamp(max=64.0), near, float(vn.abs().max()), d, softcap)
            assert ((o.view(ref.shape).double() - ref).abs() <= tol).all(), (mask, workspace is None)
