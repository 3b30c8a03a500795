"""Kernels that start before the kernel in front has ended (early_attribute),
read from their sources: each waits for it, and nothing that it reads goes
through the read-only path, which takes the data to be constant for as long as
the reading kernel is resident -- here the kernel in front may still write it."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "backward_tcgen05_tma_gemms_gb300", "csrc")


def functions():
    """(file, name) -> bodies of the free functions and methods of that name."""
    out = {}
    for f in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, f)).read()
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
        for m in re.finditer(r"\b(\w+)\s*\(", text):
            if m.group(1) in ("if", "for", "while", "switch", "return", "sizeof", "defined", "constexpr"):
                continue
            depth, i = 1, m.end()
            while depth and i < len(text):
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            head = re.match(r"\s*(const\s*)?(noexcept\s*)?\{", text[i:])
            if head is None:
                continue
            i, depth = i + head.end(), 1
            while depth and i < len(text):
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            out.setdefault((f, m.group(1)), []).append(text[m.start():i])
    return out


def reached(kernel, known):
    """The kernel and the functions that it calls, of its own file and of the headers."""
    todo, seen = [kernel], set()
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        for body in known[at]:
            own = set(re.findall(r"\bauto (\w+) = \[", body))  # lambdas
            for name in set(re.findall(r"(?<![.>\w])(\w+)\s*(?:<[^;(){}]*>)?\s*\(", body)) - own:
                todo += [k for k in known if k[1] == name and (k[0] == kernel[0] or k[0].endswith(".cuh"))]
    return seen


def test_early_kernels():
    known = functions()
    early = set()
    for (f, _), bodies in known.items():
        for body in bodies:
            if re.search(r"=\s*early_attribute\(\)", body):
                early |= {(f, k) for k in re.findall(r"cudaLaunchKernelEx\(&cfg,\s*(\w+)", body)}
    assert {k for _, k in early} >= {"sum_rows_kernel", "gemm_rows_kernel", "gemm_few_kernel"}
    for kernel in early:
        assert all("wait_for_prior_kernel()" in body for body in known[kernel]), kernel
        for at in reached(kernel, known):
            for body in known[at]:
                assert not re.search(r"__ldg\s*\(|\.nc\.|__restrict__", body), f"{kernel}: {at}"
    names = {n for _, n in reached(("gemm_rows.cu", "gemm_rows_kernel"), known)}
    assert {"rows_join_of", "linear_pre", "linear_acted", "rows_load4"} <= names
