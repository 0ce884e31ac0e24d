"""Kernels that start before their predecessor has finished wait for it on every way
out (read out of the sources: see _pdl)."""
import os
import re

import pytest

import _pdl

SOURCE = _pdl.source()
KERNELS = _pdl.overlapped_kernels(SOURCE)


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


def test_the_overlapped_kernels_are_found():
    assert {"absorb_bf16_kernel", "combine_kernel", "page_score_kernel", "split_f32_paged_kernel",
            "split_fp8_kernel", "split_pair_kernel", "split_tc_kernel"} <= set(KERNELS)


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_way_out_waits(kernel):
    assert _pdl.unwaited_exits(kernel, SOURCE) == []


def rewritten_without_barrier(kernel, read, text):
    """Whether the shared array that the statement `read` (a pattern with the array's name as
    its group) reads may be written again before every thread has read it: loops may run no
    time, so that barriers inside them count for nothing."""
    body = _pdl.body_of(kernel, text)
    m = re.search(read, body)
    rest = body[m.end():]
    while loop := re.search(r"\bwhile\s*\(", rest):
        c = _pdl.closing(rest, loop.end() - 1)
        rest = rest[:loop.start()] + rest[_pdl.statement(rest, c)[2]:]
    write = re.search(rf"\b{m.group(1)}\[[^\]]*\]\s*=(?!=)", rest)
    return bool(write) and "__syncthreads()" not in rest[:write.start()]


def test_the_choice_keeps_its_shared_words_apart():
    """With all scores equal, nothing but straight code lies between the read of the warps'
    differing bits and the counts of the ordered pass."""
    bad = "__global__ void x_kernel() { n = s[lane]; while (n) { __syncthreads(); } s[warp] = 1; }"
    assert rewritten_without_barrier("x_kernel", r"n = (\w+)\[lane\]", bad)
    good = bad.replace("} s[warp]", "} __syncthreads(); s[warp]")
    assert not rewritten_without_barrier("x_kernel", r"n = (\w+)\[lane\]", good)
    read = r"differ = (?:static_cast<uint32_t>\()?(\w+)\[lane\]"
    assert not rewritten_without_barrier("page_pick_kernel", read, SOURCE)


def test_the_header_names_what_is_read_early():
    """The selection's kernels: inputs of the caller that stand before the wait of every CTA
    that goes on are in the header's list of what is read early."""
    header = " ".join(open(os.path.join(_pdl.ROOT, "include", "mla.h")).read().split("\n * "))
    listed = re.search(r"The paged calls read (.*?) before they wait", header).group(1)
    inputs = dict(q_abs="q_abs", q_pe="q_pe", table="block_table", lengths="lengths",
                  codes="codes", scales="scales")
    helpers = dict(lengths=r"token_rows\(p,")            # reads p.lengths
    for kernel in ("select_query_kernel", "page_score_kernel", "page_pick_kernel"):
        body = _pdl.body_of(kernel, SOURCE)
        early = re.split(r"\n  pdl_wait\(\);", body)[0]    # the kernel's own wait
        assert early != body
        for field, name in inputs.items():
            if re.search(rf"\bp\.{field}\b", early) or re.search(helpers.get(field, "$^"), early):
                assert name in listed, f"{kernel} reads {name} before its wait"


@pytest.mark.parametrize("kernel", ["split_f32_paged_kernel", "split_fp8_kernel",
                                    "split_pair_kernel", "split_tc_kernel", "combine_kernel",
                                    "combine_warps_kernel"])
def test_lengths_of_a_selection_are_read_behind_a_wait(kernel):
    """Over a page selection (p.late) lengths are written by a kernel of the same call."""
    body = _pdl.body_of(kernel, SOURCE)
    first = re.search(r"\bclamp_length\(", body).start()
    assert re.search(r"if \((kPaged && )?p\.late\) pdl_wait\(\);", body[:first])
