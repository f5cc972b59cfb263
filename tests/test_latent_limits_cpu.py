"""CPU tests of the latent attention calls' limits (no kernel runs here)."""
import pytest

import rope_partial_inplace_amd as ra
from test_paged_latent_cpu import CALLS, HAS_GPU, INVALID, RUNTIME


@pytest.mark.parametrize("call", ["paged", "forward", "backward"])
def test_scales_whose_product_with_log2_e_leaves_float32_are_refused(call):
    for scale in (1e39, -1e300, 2.0 ** 128 / 1.4426, -2.0 ** 128 / 1.4426):
        assert CALLS[call]().run(scale=scale) == INVALID
        assert "scale" in ra.last_error()
    if not HAS_GPU:  # there a valid call would launch on host buffers
        for scale in (2.0 ** 126, -2.0 ** 127 * 0.99, 1e-300, -1e-45):
            assert CALLS[call]().run(scale=scale) == RUNTIME


def fake(place, dtype, *shape):
    """A contiguous tensor of that shape at an address of its own, 2^44 bytes from the next."""
    stride, n = [], 1
    for size in reversed(shape):
        stride.insert(0, n)
        n *= size
    d = ra.RopeTensor()
    d.data, d.dtype, d.ndim = (place + 1) << 44, dtype, len(shape)
    for i, size in enumerate(shape):
        d.shape[i], d.stride[i] = size, stride[i]
    return d


F32, BF16, I64 = ra.ROPE_F32, ra.ROPE_BF16, ra.ROPE_I64


def backward_of(Tq, Tk, heads, sequences):
    """Arguments of a backward call (and, by name, of a forward one) of that size, dim 64; offsets
    with sequences > 0."""
    offsets = dict(query_offsets=fake(20, I64, sequences + 1), key_offsets=fake(21, I64, sequences + 1),
                   num=0) if sequences else dict(query_offsets=None, key_offsets=None, num=1)
    return dict(offsets, query=fake(0, BF16, Tq, heads, 128), key=fake(1, BF16, Tk, heads, 64),
                key_rope=fake(2, BF16, Tk, 64), value=fake(3, BF16, Tk, heads, 64),
                out=fake(4, BF16, Tq, heads, 64), lse=fake(5, F32, Tq, heads),
                grad=fake(6, BF16, Tq, heads, 64), dquery=fake(7, BF16, Tq, heads, 128),
                dkey=fake(8, BF16, Tk, heads, 64), dkey_rope=fake(9, BF16, Tk, 64),
                dvalue=fake(10, BF16, Tk, heads, 64), workspace=12 << 44, workspace_bytes=1 << 43)


@pytest.mark.parametrize("Tq,Tk,heads,sequences,forward,backward", [
    # one-token sequences: heads * (tokens / 128 + sequences) workgroups of 256 and (dk, dv) 512 threads
    (65536, 65536, 128, 65536, True, False),
    (65536, 65536, 126, 65536, True, True),
    (1 << 20, 1 << 20, 16, 1 << 20, False, False),
    (1 << 20, 1 << 20, 15, 1 << 20, True, False),
    # many tokens and heads without offsets
    (128, 1 << 23, 128, 0, True, False),
    (128, (1 << 23) - 1024, 128, 0, True, True),
    (1 << 24, 128, 128, 0, False, False),
    ((1 << 24) - 1024, 128, 128, 0, True, True),
    # the shared key part: 16 threads a token
    (128, 1 << 28, 1, 0, True, False),
    (1 << 27, (1 << 27) - 512, 1, 0, True, True)])
def test_launches_of_2_32_threads_are_refused(Tq, Tk, heads, sequences, forward, backward):
    """Refused on the host, before anything is enqueued; sizes just below reach the launch."""
    a = backward_of(Tq, Tk, heads, sequences)
    for call, fits in (("forward", forward), ("backward", backward)):
        c = CALLS[call]()
        if not fits:
            assert c.run(**{n: v for n, v in a.items() if n in c.names}) == INVALID
            assert "too many" in ra.last_error()
        elif not HAS_GPU:
            assert c.run(**{n: v for n, v in a.items() if n in c.names}) == RUNTIME, ra.last_error()
