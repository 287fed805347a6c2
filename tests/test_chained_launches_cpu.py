"""Kernels launched while their predecessor still runs read nothing as constant data (CPU only, by the sources).

A kernel that launch_chained starts may be on the GPU before the kernel ahead of it on the stream has written its
last result, and waits for that in grid_wait.  A pointer to const with __restrict__, __ldg or ld.global.nc declares
memory that nobody writes for the whole of the kernel, and such a load may be placed ahead of the wait: in a chained
kernel that would be a race with the predecessor's writes.
"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nf4_layer_streamed_blockwise_b200", "csrc")
READ_ONLY = re.compile(r"__restrict__|__restrict\b|__ldg\s*\(|\.nc\b")


def _code(path):
    """The file without comments, string contents kept (inline PTX)."""
    src = open(path).read()
    src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
    return re.sub(r"//[^\n]*", "", src)


def _functions(src):
    """name -> (head with the parameters, body, is a kernel) of each __global__ or __device__ function."""
    out = {}
    for m in re.finditer(r"__(global|device)__", src):
        brace, semi = src.find("{", m.start()), src.find(";", m.start())
        if brace < 0 or (0 <= semi < brace):
            continue                                    # a declaration
        head = src[m.start():brace]
        flat = re.sub(r"__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)|__cluster_dims__\s*\([^()]*\)", "", head)
        name = re.search(r"([A-Za-z_]\w*)\s*\(", flat)
        if not name:
            continue                                    # a variable
        depth, i = 1, brace + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(src[i], 0)
            i += 1
        out[name.group(1)] = (flat, src[brace:i], m.group(1) == "global")
    return out


def _sources():
    return {os.path.basename(f): _code(f) for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))}


def _all_functions():
    fns = {}
    for src in _sources().values():
        fns.update(_functions(src))
    return fns


def _reached(name, fns, seen):
    """The functions of this library that a kernel's body calls, itself among them."""
    if name in seen or name not in fns:
        return seen
    seen.add(name)
    for callee in re.findall(r"\b([A-Za-z_]\w*)\s*(?:<[^;{}()]*>)?\s*\(", fns[name][1]):
        _reached(callee, fns, seen)
    return seen


def _chained():
    """Kernels that wait for a predecessor themselves or in a function they call."""
    fns = _all_functions()
    return {n: _reached(n, fns, set()) for n, (_, body, kernel) in fns.items()
            if kernel and any("grid_wait()" in fns[f][1] for f in _reached(n, fns, set()) if f != "grid_wait")}, fns


def test_the_chained_kernels_are_found():
    """Every kernel handed to launch_chained, by the call or through a chosen variable, waits for its predecessor."""
    chained, fns = _chained()
    kernels = {n for n, f in fns.items() if f[2]}
    named = set()
    for src in _sources().values():
        if "launch_chained(" not in src:
            continue
        # the kernels of a file that launches chained: all of them are launched so
        named |= {n for n in kernels if re.search(rf"__global__[^;{{]*\b{n}\s*\(", src)}
    assert len(named) >= 10
    assert named == set(chained), named ^ set(chained)


def test_chained_kernels_load_nothing_as_constant():
    chained, fns = _chained()
    bad = []
    for kernel, reached in chained.items():
        for f in sorted(reached):
            head, body, _ = fns[f]
            for where, text in (("parameters", head), ("body", body)):
                if READ_ONLY.search(text):
                    bad.append((kernel, f, where, READ_ONLY.search(text).group(0)))
    assert not bad, bad


def test_chained_kernels_wait_before_global_memory():
    """In the body that holds the wait, nothing ahead of it dereferences an argument: only shared memory, barriers and
    tensor memory are set up."""
    chained, fns = _chained()
    holders = {f for reached in chained.values() for f in reached if "grid_wait()" in fns[f][1] and f != "grid_wait"}
    assert len(holders) >= 10
    for f in sorted(holders):
        head, body, _ = fns[f]
        ahead = body[:body.index("grid_wait()")]
        for p in re.findall(r"([A-Za-z_]\w*)\s*(?:,|\)|$)", head[head.index("("):]):
            assert not re.search(rf"\b{p}(?:\.\w+)*\s*\[", ahead), (f, p)
        assert not re.search(r"tma_load|bulk_g2s|atomic|ln_fetch|epi_fetch", ahead), f
