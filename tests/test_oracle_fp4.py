"""Pins of the oracle's 4-bit quantiser: landmark values and ties by hand,
brute force, torch's E4M3 cast for the scales, and the refusals of the 4-bit
and chunk-list calls that need no GPU."""
import ctypes as C

import numpy as np
import pytest

from oracle import fp4


@pytest.mark.parametrize("y,v", [
    (0.0, 0.0), (0.25, 0.0), (0.2500001, 0.5), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (2.6, 3.0),
    (3.5, 4.0), (5.0, 4.0), (5.01, 6.0), (7.0, 6.0), (1e9, 6.0), (-1.25, -1.0), (-1.75, -2.0), (-6.4, -6.0)])
def test_e2m1_landmarks_and_ties(y, v):
    assert fp4.nearest_e2m1([y])[0] == v


def test_blocks_by_hand():
    # a block whose largest value is 6: scale 1, values on the grid stay
    x = np.zeros((1, 16), np.float16)
    x[0, :8] = [6, -4, 3, 2, 1.5, 1, 0.5, -0.5]
    c, s = fp4.quantize(x, 1.0)
    assert s.tolist() == [[1.0]] and (c == x).all()
    # under S = 2 the same block halves its scale and reads back the same
    c, s = fp4.quantize(x, 2.0)
    assert s.tolist() == [[0.5]] and (fp4.dequantize(c, s, 2.0) == x).all()
    # nothing but zeros: scale 0, codes 0
    c, s = fp4.quantize(np.zeros((1, 32), np.float16), 1.0)
    assert (c == 0).all() and (s == 0).all()
    # below half of the smallest scale (2^-10 * 6): the block is lost as zeros
    c, s = fp4.quantize(np.full((1, 16), 2.0 ** -10 * 6 * 0.9, np.float16), 1.0)
    assert (s == 0).all() and (c == 0).all()
    # beyond 448 * 6 the scale saturates and the codes with it
    c, s = fp4.quantize(np.full((1, 16), 60000, np.float16), 1.0)
    assert (s == 448).all() and (c == 6).all()


def test_against_torch_and_brute_force():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((64, 128)) * np.exp2(rng.integers(-12, 9, (64, 1)))).astype(np.float16)
    c, s = fp4.quantize(x, 0.37)
    y = torch.from_numpy(x).float() * float(np.float32(1) / np.float32(0.37))
    top = y.reshape(64, 8, 16).abs().amax(-1) * float(np.float32(1) / np.float32(6))
    ts = top.clamp(max=448).to(torch.float8_e4m3fn).float()
    np.testing.assert_array_equal(s, ts.numpy().astype(np.float64))
    z = y.reshape(64, 8, 16) * torch.where(ts > 0, 1 / ts, torch.zeros(()))[..., None]
    grid = torch.tensor(np.concatenate([-fp4.VALUES[::-1], fp4.VALUES]))
    d = (z.double()[..., None] - grid).abs()
    np.testing.assert_array_equal((torch.from_numpy(c).reshape(64, 8, 16) - z.double()).abs().numpy(), d.amin(-1).numpy())
    # what the tensor cores multiply is exact in fp16
    v = fp4.stored(c, s)
    np.testing.assert_array_equal(v, v.astype(np.float16).astype(np.float64))


def test_fp4_pool_shapes_and_refusals(lib):
    from prefix_shared_decode_gb300 import CAError, Pool, capi
    p = Pool(2, 4, 128, 64, 10, host_only=True, kv_dtype="fp4", n_kv_heads=2)
    tile = 2 * (64 * 128 // 2 + 64 * 128 // 16)
    assert p.kv_bytes == 10 * 2 * 2 * tile + 256
    b = Pool(2, 4, 128, 64, 10, host_only=True, kv_dtype="fp4", n_kv_heads=2, chunk_bounds=True)
    assert b.kv_bytes == p.kv_bytes + 10 * 2 * 2 * 2 * 128 * 2
    assert Pool(1, 2, 64, 16, 10, host_only=True, kv_dtype="fp4").kv_bytes == 10 * 2 * 1152 + 256
    for bad, name in [(dict(head_dim=256, chunk=32), "CA_ERR_UNSUPPORTED"), (dict(k_scale=-1.0), "CA_ERR_INVALID"),
                      (dict(v_scale=float("nan")), "CA_ERR_INVALID"), (dict(v_scale=float("inf")), "CA_ERR_INVALID"),
                      (dict(chunk=48), "CA_ERR_UNSUPPORTED")]:
        kw = dict(n_layers=1, n_heads=2, head_dim=128, chunk=16, capacity_slots=4, host_only=True, kv_dtype="fp4")
        kw.update(bad)
        with pytest.raises(CAError) as e:
            Pool(**kw)
        assert e.value.name == name, bad
    with pytest.raises(ValueError):
        Pool(1, 2, 128, 16, 4, host_only=True, kv_dtype="int4")
    n = C.c_size_t()
    both = capi.PoolConfig(1, 2, 128, 16, 4, capi.CA_KV_FP8 | capi.CA_KV_FP4)
    assert lib.ca_pool_bytes(C.byref(both), C.byref(n)) == -1
    unknown = capi.PoolConfig(1, 2, 128, 16, 4, 16)
    assert lib.ca_pool_bytes(C.byref(unknown), C.byref(n)) == -1


def test_chunk_list_calls_refuse_without_a_device(lib):
    from prefix_shared_decode_gb300 import CAError, Pool, select_chunks, sparse_decode_attention
    p = Pool(1, 2, 64, 16, 8, host_only=True, chunk_bounds=True)
    p.insert(1, list(range(40)))
    assert p.seq_len(1) == 40
    with pytest.raises(CAError) as e:
        p.seq_len(2)
    assert e.value.name == "CA_ERR_NOT_FOUND"
    s = p.schedule([1], chunk_lists=True)
    plain = p.schedule([1])
    with pytest.raises(ValueError):
        p.read(1)
    with pytest.raises(ValueError):
        select_chunks(p, s, None, 2)
    with pytest.raises(ValueError):
        sparse_decode_attention(p, s, None, None)
    buf = (C.c_uint8 * 64)()
    a = (C.addressof(buf) + 15) // 16 * 16
    ids = (C.c_int64 * 1)(1)
    ln = (C.c_int32 * 1)(1)
    # a host-only pool, NULL objects
    assert lib.ca_select_chunks(p.handle, s.handle, 0, a, 2, 1, 1, a, None) == -1
    assert lib.ca_sparse_attention(p.handle, s.handle, 0, a, a, 2, a, 1.0, None) == -1
    assert lib.ca_select_chunks(None, s.handle, 0, a, 2, 1, 1, a, None) == -1
    assert lib.ca_sparse_attention(p.handle, None, 0, a, a, 2, a, 1.0, None) == -1
    assert lib.ca_read_batch(p.handle, 1, ids, None, ln, a, a, None) == -1
    assert lib.ca_read_batch(None, 1, ids, None, ln, a, a, None) == -1
    assert lib.ca_seq_lengths(p.handle, 1, ids, None) == -1
    assert lib.ca_seq_lengths(p.handle, 1, None, ln) == -1
    assert lib.ca_seq_lengths(p.handle, 1, (C.c_int64 * 1)(7), ln) == -3
    # the lists change nothing in the tables, and a schedule is rebuilt when the flag changes
    for k, v in s.tables().items():
        np.testing.assert_array_equal(v, plain.tables()[k])
    again = p.schedule([1], reuse=s)
    assert again is s and again.counts() == plain.counts()
