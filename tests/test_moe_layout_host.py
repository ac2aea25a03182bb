"""The shared memory of a CTA of the moe kernel, without a GPU: for every number
of tokens and every cut of the k blocks, what the kernel may read lies inside
its allocation."""
import pytest

# k blocks of 128 on either side, whole and ragged, up to the widest
SIZES = [16, 112, 128, 144, 640, 768, 784, 1024, 1280, 1552, 2048, 2064, 3840, 4096, 5120, 6144, 7168, 8192, 8208,
         10000, 12288, 14000, 15872, 15888, 16000, 16384]


@pytest.fixture(scope="module")
def capi():
    from mhc_residual_boundary_gb300 import build
    build.build()
    from mhc_residual_boundary_gb300 import capi as c
    c.lib()
    return c


def widths(m):
    """The tokens whose sums a warp takes for an expert of 1 to m of them."""
    return {5 if n <= 5 else 10 if n <= 10 else 32 for n in range(1, m + 1)}


@pytest.mark.parametrize("sms", [148, 152, 160])
@pytest.mark.parametrize("fp8", [True, False])
def test_every_read_lies_inside(capi, sms, fp8):
    pieces = (3, 2)[not fp8]
    for hidden in SIZES:
        for intermediate in SIZES:
            for top_k, shared in ((1, 0), (8, 1), (16, 8)):
                config = capi.mhc_sublayer_config_t(hidden, intermediate, 64, shared, top_k, 32, 0, 1.0,
                                                    capi.MHC_SUBLAYER_FP8 if fp8 else 0)
                for m in range(1, 33):
                    f = capi.mhc_test_moe_form(config, m, sms)
                    what = (hidden, intermediate, top_k, shared, m)
                    assert f.stages >= 2 and f.ring_at % 1024 == 0 and f.stage_bytes % 1024 == 0, what
                    # the rows of an expert's tokens, and those that an MMA reads, its
                    # columns a multiple of 16
                    rows = m * pieces
                    assert f.weight_bytes + rows * 128 <= f.stage_bytes, what
                    last = f.ring_at + (f.stages - 1) * f.stage_bytes + f.weight_bytes
                    end = last + (rows + 15) // 16 * 16 * 128
                    assert end <= f.size, what
                    if fp8:
                        assert f.ring_at + f.stages * f.stage_bytes <= f.scales_at, what
                        first = (f.items * f.scale_blocks - 1) * m   # the last block's
                        assert f.scales_at + 4 * (first + max(widths(m))) <= f.size, what
                        assert f.scale_blocks <= 32, what            # a block a lane


def test_the_hook_refuses_what_no_call_has(capi):
    good = (256, 128, 8, 1, 2, 4, 0, 1.0, capi.MHC_SUBLAYER_FP8)
    capi.mhc_test_moe_form(capi.mhc_sublayer_config_t(*good), 4, 152)
    for config, m, sms in ((good, 0, 152), (good, 33, 152), (good, 4, 0), ((0,) + good[1:], 4, 152),
                           (good[:4] + (0,) + good[5:], 4, 152)):
        with pytest.raises(capi.MhcError, match="MHC_ERR_INVALID_ARG"):
            capi.mhc_test_moe_form(capi.mhc_sublayer_config_t(*config), m, sms)
