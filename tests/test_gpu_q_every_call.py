"""GPU: calls in a row, and on two streams at once: the result of every one of
them, bit for bit, so that a race that spoils one call in many is seen."""
import pytest
import torch

from tests.test_gpu_l_attn_bwd import both, bsa, make, random_lists  # noqa: F401

pytestmark = pytest.mark.gpu

BITS = {torch.bfloat16: torch.int16, torch.float32: torch.int32, torch.int32: torch.int32}


def differs(ref, got):
    """Device flag: some bit of the tensors differs."""
    flag = torch.zeros((), dtype=torch.bool, device="cuda")
    for a, b in zip(ref, got, strict=True):
        flag |= (a.view(BITS[a.dtype]) != b.view(BITS[b.dtype])).any()
    return flag


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["frames", "lists", "few"])
def test_every_gradient(bsa, kind, d):  # noqa: F811
    """Masks in every tile; lists; rows of few keys, some of them of one."""
    if kind == "frames":
        T, N, H = 21, 21 * 157, 4
        frames, counts, _ = bsa.lvsa_build_index(T, 5, 3, 7, 0, device="cuda")
        ix = bsa.lvsa_index(T, frames, counts)
    else:
        N, H = (2000, 3) if kind == "lists" else (8 * 128 + 1, 3)
        ix = bsa.block_index(*random_lists(H, -(-N // 128), 0.4, 8))
    go, q, k, v = make(N, H, d, seed=85)
    o, lse, ref = both(bsa, go, q, k, v, ix)
    flags = []
    for _ in range(6):                                       # calls back to back, then their comparison
        got = [bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix) for _ in range(50)]
        flags += [differs(ref, x) for x in got]
    assert bsa.get_device_status() == bsa.BSA_OK
    assert torch.stack(flags).nonzero().flatten().tolist() == []


@pytest.mark.parametrize("d", [64, 128])
def test_every_forward_and_choice(bsa, d):  # noqa: F811
    N, H = 21 * 157, 4
    _, q, k, v = make(N, H, d, seed=86)
    ix = bsa.block_index(*bsa.blockmean_select(q, k, 9, 1))
    call = lambda: (*bsa.blockmean_select(q, k, 9, 1), *bsa.blocksparse_attn_fwd(q, k, v, ix))   # noqa: E731
    ref = call()
    flags = []
    for _ in range(4):
        got = [call() for _ in range(50)]
        flags += [differs(ref, x) for x in got]
    assert bsa.get_device_status() == bsa.BSA_OK
    assert torch.stack(flags).nonzero().flatten().tolist() == []


def test_every_chain_on_two_streams(bsa):  # noqa: F811
    N, H, d = 3000, 4, 128
    g = torch.Generator(device="cuda").manual_seed(95)
    x = [torch.randn((N, 3, H, d), generator=g, device="cuda").bfloat16() for _ in range(2)]
    go = torch.randn((N, H, d), generator=g, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    rope = bsa.rope_axes([bsa.rope_build_table(n, p, device="cuda") for n, p in zip((30, 10, 10), (22, 21, 21))],
                         grid=(30, 10, 10))

    def chain(x, stream):
        with torch.cuda.stream(stream):
            v = x[:, 2].contiguous()
            q, k = bsa.qk_norm_rope_fwd(x[:, 0], x[:, 1], w, w, rope)
            idx, cnt = bsa.blockmean_select(q, k, 6, 1)
            o, lse, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
            back = bsa.qk_norm_rope_bwd(grads[0], grads[1], x[:, 0], x[:, 1], w, w, rope)
            return (q, k, idx, cnt, o, lse, *grads, *back)

    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    ref = []
    for i in range(2):
        ref.append(chain(x[i], streams[i]))
        torch.cuda.synchronize()
    rounds = [[chain(x[i], streams[i]) for i in range(2)] for _ in range(20)]      # all results are kept
    torch.cuda.synchronize()
    assert bsa.get_device_status() == bsa.BSA_OK
    flags = [differs(ref[i], r[i]) for r in rounds for i in range(2)]
    assert torch.stack(flags).nonzero().flatten().tolist() == []
