"""When the build makes the extension anew: it binds to one torch's C++ classes."""
import os

from backward_tcgen05_tma_gemms_gb300 import build


def test_extension_follows_torch(monkeypatch, tmp_path):
    lib, binding, stamp = (str(tmp_path / n) for n in ("lib.so", "_binding.so", "binding.txt"))
    for name, path in (("LIB", lib), ("BINDING", binding), ("BINDING_STAMP", stamp)):
        monkeypatch.setattr(build, name, path)
    open(lib, "w").close()
    monkeypatch.setattr(build, "_deps_mtime", lambda: os.path.getmtime(lib))
    made = []

    def compiled():
        made.append(1)
        open(binding, "w").close()
        with open(stamp, "w") as f:
            f.write(build._torch_stamp())
    monkeypatch.setattr(build, "_compile_binding", compiled)
    assert build.build() == lib and len(made) == 1      # there was none
    assert build.build() == lib and len(made) == 1      # unchanged
    import torch
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert build.build() == lib and len(made) == 2      # another torch, the same sources
    assert build.build() == lib and len(made) == 2
    os.remove(stamp)
    assert build.build() == lib and len(made) == 3      # of an unknown torch
    os.utime(binding, (0, 0))
    assert build.build() == lib and len(made) == 4      # older than the sources
    assert build.build() == lib and len(made) == 4
