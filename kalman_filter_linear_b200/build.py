"""Build libkdn.so in-tree with nvcc for sm_100a.

    python -m kalman_filter_linear_b200.build

The library is a plain shared object with a C ABI (include/kdn.h); it links
only the CUDA runtime.  Output: kalman_filter_linear_b200/libkdn.so, and beside it
_kdn_quick.so, the quick form of the binding's small calls, which is built against
torch's headers (without them the binding goes through ctypes alone).
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, 'libkdn.so')
QUICK = os.path.join(PKG, '_kdn_quick.so')
ARCH = ['-gencode', 'arch=compute_100a,code=sm_100a']


def nvcc():
    for cand in (os.environ.get('NVCC'), shutil.which('nvcc'), '/usr/local/cuda/bin/nvcc'):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError('nvcc not found')


def sources():
    return sorted(glob.glob(os.path.join(PKG, 'csrc', '*.cu')))


def build(verbose=False, extra=()):
    """Compile every source to an object in parallel, then link the library."""
    from concurrent.futures import ThreadPoolExecutor
    srcs = sources()
    objdir = os.path.join(ROOT, '_build')
    os.makedirs(objdir, exist_ok=True)
    flags = ['-Xcompiler', '-fPIC', '-O3', '-lineinfo', '-std=c++17', *ARCH,
             '-I', os.path.join(ROOT, 'include'), '--expt-relaxed-constexpr',
             '-Xptxas', '-warn-spills', *extra]

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + '.o')
        cmd = [nvcc(), '-c', *flags, '-o', obj, src]
        if verbose:
            print(' '.join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, srcs))
    subprocess.run([nvcc(), '-shared', *ARCH, '-o', LIB + '.tmp', *objs, '-lcudart'], check=True)
    os.replace(LIB + '.tmp', LIB)
    build_quick(verbose)
    return LIB


def quick_sources():
    return [os.path.join(PKG, 'csrc', 'quick_binding.cpp'), os.path.join(ROOT, 'include', 'kdn.h')]


def quick_command():
    """The command that compiles _kdn_quick.so, or None without torch or g++."""
    spec = importlib.util.find_spec('torch')
    cxx = shutil.which('g++')
    if spec is None or cxx is None:
        return None
    torch = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return [cxx, '-O2', '-std=c++17', '-fPIC', '-shared', '-I', os.path.join(torch, 'include'),
            '-I', os.path.join(torch, 'include', 'torch', 'csrc', 'api', 'include'),
            '-I', os.path.join(cuda, 'include'), '-I', sysconfig.get_paths()['include'],
            quick_sources()[0], '-o', QUICK + '.tmp', '-L', PKG,
            '-l:libkdn.so', '-L', os.path.join(torch, 'lib'), '-lc10', '-lc10_cuda', '-ltorch',
            '-ltorch_cpu', '-ltorch_python', '-Wl,-rpath,$ORIGIN']


def build_quick(verbose=False):
    """Compile _kdn_quick.so; without it the binding works the same, slower."""
    cmd = quick_command()
    if os.path.exists(QUICK):
        os.remove(QUICK)
    if cmd is None:
        return
    if verbose:
        print(' '.join(cmd), flush=True)
    if subprocess.run(cmd).returncode == 0:
        os.replace(QUICK + '.tmp', QUICK)
    else:
        print('_kdn_quick.so could not be built: calls go through ctypes', file=sys.stderr)


def quick_is_stale():
    """Whether _kdn_quick.so is missing or older than its sources, and could be built."""
    if os.path.exists(QUICK) and \
            os.path.getmtime(QUICK) >= max(os.path.getmtime(d) for d in quick_sources()):
        return False
    return quick_command() is not None


def is_stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(PKG, 'csrc', '*.cuh')) + \
        glob.glob(os.path.join(PKG, 'csrc', '*.h')) + glob.glob(os.path.join(ROOT, 'include', '*.h'))
    return any(os.path.getmtime(d) > t for d in deps) or quick_is_stale()


if __name__ == '__main__':
    extra = sys.argv[1:]
    print(build(verbose=True, extra=extra))
