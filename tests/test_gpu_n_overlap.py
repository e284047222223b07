"""GPU: outputs of the rotation calls next to tensors in the same buffer: interleaved
slices work in place, shared memory is refused and nothing is written."""
import pytest
import torch

from tests.test_gpu_j_rope import bsa, make, setup  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", ["N3Hd", "NH3d", "3HNd", "HN3d", "H3Nd"])
def test_slices_in_place(bsa, order):  # noqa: F811
    N, H, d = 60, 3, 64
    r, _ = setup(bsa, (3, 4, 5), 0, d, False)
    sizes = {"N": N, "3": 3, "H": H, "d": d}
    room = make((N * 3, H, d), torch.bfloat16, "whole", 1).reshape([sizes[c] for c in order])
    at = order.index("3")
    rest = order.replace("3", "")

    def slices(t):
        return [t.select(at, i).permute([rest.index(c) for c in "NHd"]) for i in range(3)]

    w = 1 + 0.1 * torch.arange(d, device="cuda") / d
    q, k, v = (x.contiguous() for x in slices(room))
    qo, ko = bsa.qk_norm_rope_fwd(q, k, w, w, r)
    gq, gk = make((N, H, d), torch.bfloat16, "whole", 2), make((N, H, d), torch.bfloat16, "whole", 3)
    dq, dk, dwq, dwk = bsa.qk_norm_rope_bwd(gq, gk, q, k, w, w, r)
    a = room.clone()
    sq, sk, sv = slices(a)
    bsa.qk_norm_rope_fwd(sq, sk, w, w, r, qo=sq, ko=sk)
    assert torch.equal(sq, qo) and torch.equal(sk, ko) and torch.equal(sv, v)
    a = room.clone()
    sq, sk, sv = slices(a)
    got = bsa.qk_norm_rope_bwd(gq, gk, sq, sk, w, w, r, dq=sq, dk=sk)
    assert torch.equal(sq, dq) and torch.equal(sk, dk) and torch.equal(sv, v)
    assert torch.equal(got[2], dwq) and torch.equal(got[3], dwk)


def test_refusals(bsa):  # noqa: F811
    r, _ = setup(bsa, (3, 4, 5), 0, 64, False)
    room = make((200, 4, 64), torch.bfloat16, "whole", 4)
    keep = room.clone()
    x, g, k = room[:60], room[60:120], room[120:180]
    calls = [lambda: bsa.rope_apply(x, r, out=room[1:61]),
             lambda: bsa.rope_apply(room[:60, :4].reshape(60, 4, 64), r, out=room[30:90]),
             lambda: bsa.rope_apply(room[:4, :4], bsa.rope_axes([bsa.rope_build_table(1, 4)], grid=(1,)),
                                    out=room[:4].transpose(0, 1)),
             lambda: bsa.qk_norm_rope_fwd(x, k, qo=k),
             lambda: bsa.qk_norm_rope_fwd(x, k, qo=g, ko=g),
             lambda: bsa.qk_norm_rope_bwd(g, x, x, k, dq=k),
             lambda: bsa.qk_norm_rope_bwd(g, k, x, k, dk=x),
             lambda: bsa.qk_norm_rope_bwd(x, x, g, g, dq=k, dk=k)]
    for call in calls:
        with pytest.raises(bsa.BsaError):
            call()
    assert torch.equal(room, keep) and bsa.get_device_status() == bsa.BSA_OK
