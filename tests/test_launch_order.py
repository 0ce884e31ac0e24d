"""Kernels that start before their predecessor has finished wait for it on every way
out (read out of the sources: see _pdl)."""
import pytest

import _pdl

SOURCE = _pdl.source()


def test_the_reading_finds_missing_waits():
    """The reader itself: what it takes for a wait, and what not."""
    def exits(body):
        return _pdl.unwaited_exits("x_kernel", f"__global__ void x_kernel(int n) {{ {body} }}")

    assert exits("pdl_wait(); if (n) return;") == []
    assert exits("if (n) return; pdl_wait();") == ["return"]
    assert exits("if (p.late) pdl_wait(); n = 1;") == ["end"]
    assert exits("if (p.late) pdl_wait(); pdl_wait();") == []
    assert exits("if (tid == 0) pdl_wait(); __syncthreads();") == []
    assert exits("if (warp == 8) { n = 1; } else if (kShare && warp < 3) { pdl_wait(); }") == []
    assert exits("for (int i = 0; i < n; ++i) { pdl_wait(); }") == ["end"]
    assert exits("if (n) { pdl_wait(); } else { pdl_wait(); }") == []
    assert exits("if (r0 >= n) { if (r0 == 0) pdl_wait(); return; } pdl_wait();") == []
    assert exits("if (r0 >= n) { if (p.direct || r0 == 0) pdl_wait(); return; } pdl_wait();") == []
    assert exits("if (r0 >= n) { if (r0 == 0 && n) pdl_wait(); return; } pdl_wait();") == ["return"]
    assert exits("auto f = [&] { return 1; }; pdl_wait(); f();") == []
    found = _pdl.overlapped_kernels("launch_pdl(n ? a_kernel<1> : b_kernel<2>, dim3(1), p);")
    assert found == ["a_kernel", "b_kernel"]


@pytest.mark.parametrize("kernel", ["split_f32_paged_kernel", "page_score_kernel"])
def test_every_way_out_waits(kernel):
    assert kernel in _pdl.overlapped_kernels(SOURCE)
    assert _pdl.unwaited_exits(kernel, SOURCE) == []
