"""The 8-bit key/value row calls where they could go wrong, on the CPU."""
import ctypes
import os
import subprocess

import pytest
import torch

import sparse_attention_kv_swap_gb300 as pkg
from sparse_attention_kv_swap_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_kv_swap_gb300 import build
    build.build()
    return B.load_library()


def cpu_cache(R=3, L=40, W=256, layers=2):
    """A cache without a handle, its tensors in host memory: a call that is refused on the
    host needs no more."""
    from sparse_attention_kv_swap_gb300.cache import SwapInCache
    cache = SwapInCache.__new__(SwapInCache)
    cache.cfg = pkg.make_config(R, L, W, 16, 8, 1, num_layers=layers)
    cache.device = torch.device("cpu")
    cache.host_pools = [torch.zeros((R, L, W), dtype=torch.uint8) for _ in range(layers)]
    cache.device_kv = [torch.zeros((R * 24, W), dtype=torch.uint8) for _ in range(layers)]
    return cache


def evict_refusals(make):
    """(arguments of evict that a cache of 3 requests of 40 tokens in 2 layers refuses), each from
    fresh scales and sums of make(shape)."""
    fmt = pkg.make_kv_format(2, 64, 16)
    good = dict(requests=[0, 2], seq_lens=[40, 30], budget=8, recent=2)

    def scales(R=3, blocks=3, n=2):
        return [make((R, blocks, 2, 2)) for _ in range(n)]

    def acc(R=3, L=40, n=2):
        return [make((R, L)) for _ in range(n)]

    bad = [dict(requests=[0, -1]), dict(requests=[0, 3]), dict(requests=[2, 2]),
           dict(requests=[1 << 40, 0]), dict(requests=[0]), dict(seq_lens=[40, 41]),
           dict(seq_lens=[-1, 0]), dict(budget=0, recent=0), dict(recent=9), dict(recent=-1),
           dict(scales=scales(n=1)), dict(scales=scales(n=3)), dict(scales=scales(blocks=2)),
           dict(scales=scales(R=2)), dict(scales=[x.half() for x in scales()]),
           dict(scales=[x.transpose(0, 2).contiguous().transpose(0, 2) for x in scales()]),
           dict(acc=acc(n=1)), dict(acc=acc(L=39)), dict(acc=acc(R=4)),
           dict(acc=[x.double() for x in acc()]), dict(acc=[acc(n=1)[0], acc(L=41, n=1)[0]]),
           dict(fmt=pkg.make_kv_format(1, 64, 16)),  # narrower rows than the cache's
           dict(fmt=pkg.HsKvFormat(1, 100, 16, pkg.HS_KV_E4M3, 256))]  # no such head size
    for kw in bad:
        yield {**dict(fmt=fmt, scales=scales(), acc=acc()), **good, **kw}


def test_cache_evict_refuses_on_the_host(lib):
    cache = cpu_cache()
    for kw in evict_refusals(torch.ones):
        with pytest.raises(ValueError):
            cache.evict(**kw)


def test_cache_evict_refuses_pools_of_another_shape(lib):
    kw = next(evict_refusals(torch.ones))
    kw["requests"] = [0, 2]
    cache = cpu_cache()
    for pool in (cache.host_pools[1].view(-1), cache.host_pools[1].view(torch.int8)):
        cache.host_pools[1] = pool
        with pytest.raises(ValueError, match="host pools"):
            cache.evict(**kw)


def run_cuda_program(name, tmp_path):
    """Compiles tests/c/<name>.cu, which needs no GPU, and returns what it prints."""
    from sparse_attention_kv_swap_gb300 import build
    try:
        nvcc = build._nvcc()
    except Exception:
        pytest.skip("no nvcc")
    exe = str(tmp_path / name)
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", name + ".cu")
    cmd = ([nvcc] + build.ARCH_FLAGS + build.NVCC_FLAGS
           + ["-I", build.INCLUDE, "-I", build.CSRC, src, "-o", exe])
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    return res.stdout


def test_attend_shapes_fit_an_sm(tmp_path):
    """Every head size, head layout and length that hs_attend accepts gets a launch shape that
    an SM can run."""
    assert run_cuda_program("attend_shapes", tmp_path).startswith("ok ")


def test_a_failed_launch_leaves_no_error_behind(tmp_path):
    assert run_cuda_program("kv_errors", tmp_path).startswith("ok")


def test_compact_refuses_overlapping_scales(lib):
    """Scales that source and destination share would be read and written in any order."""
    fmt = pkg.make_kv_format(8, 128, 64)
    at, src, dst = 0x20000, 0x1000000, 0x2000000
    scales = 0x400000  # of 2 requests with 3 blocks of 2 x 8 floats: 384 bytes

    def call(dst_scales):
        return lib.hs_compact_kv(ctypes.byref(fmt), src, scales, 2, 130, at, at, at, 1, 32, dst,
                                 dst_scales, 2, 70, at, None)

    # the destination's 2 requests with 2 blocks: 256 bytes
    for to in (scales, scales + 380, scales - 252, scales + 64):
        assert call(to) == B.HS_ERR_INVALID_ARG, hex(to)


@pytest.mark.parametrize("layer", [-1, -2, 2])
def test_cache_attend_refuses_layers_out_of_range(lib, layer):
    """As every other call of the cache does; -1 is not its last layer."""
    cache, fmt = cpu_cache(), pkg.make_kv_format(2, 64, 16)
    topk = torch.zeros((1, 1, 8), dtype=torch.int32)
    with pytest.raises(pkg.HsError) as error:
        cache.attend(fmt, torch.ones((3, 3, 2, 2)), torch.zeros((1, 1, 4, 64)).bfloat16(), topk, topk,
                     topk[:, 0, 0], layer_id=layer)
    assert error.value.code == B.HS_ERR_INVALID_ARG
