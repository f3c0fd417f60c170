"""Checks of the Python binding of the NVFP4 cache, scored attention and the
adapters that need no GPU: the cache's descriptor and its refusals."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv


def caches(nb=4, page=16, heads=2, D=64, order="nhd"):
    def one(n):
        if order == "hnd":
            return torch.zeros(nb, heads, page, n, dtype=torch.uint8).transpose(1, 2)
        return torch.zeros(nb, page, heads, n, dtype=torch.uint8)
    g = torch.ones(1)
    return (one(D // 2), one(D // 16), g), (one(D // 2), one(D // 16), g)


def strides(c):
    return (c.stride_block, c.stride_token, c.stride_head, c.scale_stride_block,
            c.scale_stride_token, c.scale_stride_head)


def test_descriptor():
    c = nv._kv_cache4(*caches())
    assert (c.num_blocks, c.page, c.n_kv_heads, c.D) == (4, 16, 2, 64)
    assert strides(c) == (1024, 64, 32, 128, 8, 4)
    assert strides(nv._kv_cache4(*caches(order="hnd"))) == (1024, 32, 512, 128, 4, 64)
    # a dimension of one: any stride that the library takes
    for shape in ((1, 16, 2), (4, 1, 2), (4, 16, 1), (1, 1, 1)):
        for D in (64, 128, 192):
            c = nv._kv_cache4(*caches(*shape, D=D))
            s = strides(c)
            assert all(x >= D // 2 and x % 16 == 0 for x in s[:3])
            assert all(x >= D // 16 and x % 4 == 0 for x in s[3:])
    a, b = caches(4, 16, 1), caches(4, 16, 1, order="hnd")
    assert a[0][0].stride() != b[0][0].stride()
    assert strides(nv._kv_cache4(a[0], b[1])) == strides(nv._kv_cache4(*a))


def test_descriptor_refusals():
    k, v = caches()
    with pytest.raises(TypeError):
        nv._kv_cache4((k[0].to(torch.int8), k[1], k[2]), v)
    with pytest.raises(TypeError):
        nv._kv_cache4(k, (v[0], v[1].float(), v[2]))
    with pytest.raises(TypeError):
        nv._kv_cache4((k[0], k[1], torch.ones(2)), v)
    with pytest.raises(TypeError):
        nv._kv_cache4((k[0], k[1], torch.ones(1).double()), v)
    with pytest.raises(ValueError):
        nv._kv_cache4((k[0], k[1][..., :3], k[2]), (v[0], v[1][..., :3], v[2]))
    with pytest.raises(ValueError):
        nv._kv_cache4(k, caches(nb=3)[1])
    with pytest.raises(ValueError):
        nv._kv_cache4(*caches(D=32))
    with pytest.raises(ValueError, match="strides"):
        nv._kv_cache4(k, caches(order="hnd")[1])
    wide = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)[..., ::2]
    with pytest.raises(ValueError, match="strides"):
        nv._kv_cache4((wide, k[1], k[2]), (wide, v[1], v[2]))


def test_scores():
    assert nv._scores(0.0, None, 4) is None
    with pytest.raises(ValueError, match="slopes"):
        nv._scores(0.0, torch.ones(3), 4)
    with pytest.raises(ValueError, match="slopes"):
        nv._scores(0.0, torch.ones(4).double(), 4)
    with pytest.raises(ValueError, match="slopes"):
        nv._scores(0.0, torch.ones(8)[::2], 4)


def test_what_is_not_on_a_device_is_refused():
    k, v = caches()
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        nv.paged_attention_nvfp4(q, k, v, t, n)
    with pytest.raises(ValueError, match="device"):
        nv.rope_append_nvfp4(None, q, q, torch.zeros(1).long(), torch.zeros(1).long(),
                             torch.ones(32), k, v)
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        nv.lora_segments([(a, b)], torch.zeros(1, 64, dtype=torch.bfloat16), n)
    with pytest.raises(ValueError, match="length"):
        nv.lora_segments_into([], q, n, [], n)
