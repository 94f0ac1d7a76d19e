"""How the report of registers names kernels."""
from depthwise_convolution_amd import _build


def test_kernel_names():
    name = _build._kernel_name
    hidden = "(anonymous namespace)::"
    assert name(f"dwseq::{hidden}k_db(float const*, int, int, float*)") == "k_db"
    assert name(f"void dwmix::{hidden}k_walk<half, 128, 64, 1, (dwmix::{hidden}Mode)2>"
                "(dwmix::Walks)") == "void k_walk<_Float16, 128, 64, 1, ODD>"
    assert name(f"void dwseq::{hidden}k_gemm_256<dwseq::I8<__int128>, false, false>"
                "(dwseq::Product, int, int, int)") == "void k_gemm_256<I8<__bf16>, false, false>"
    assert name(f"void dwconv::{hidden}k_tiled_nhwc<3, 3>(dwconv::Args)") == \
        "void k_tiled_nhwc<3, 3>"
