"""The compiled binding of the 8-bit cache's and the rotary calls: arguments of the wrong kind or
size are exceptions, never another value. No GPU is needed."""
import ctypes
import importlib.util
import sysconfig

import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build

# Calls that have nothing to do (status 0), and the C type of each argument.
CACHE = pk._PaQ8Cache(16, 16, 16, 16, 1)
ROTARY = pk._PaRotary(16, 16, 128, 1, 0, 1.0)
A, R = ctypes.addressof(CACHE), ctypes.addressof(ROTARY)
HEAD, TAIL = [16, 16, 16, 16, 2048, 2048, 1024, 1024, 1, 16, 0, R], [16, 0, 16, 8, 128, 16, 4, None, None]
CALLS = {
    "pa_store_kvcache_q8": ([16, 16, 1024, 1024, 1, A, 16, 0, 8, 128, 16, 4, None, None],
                            "ppllippiiiilpp"),
    "pa_load_kvcache_q8": ([16, 16, 1, A, 16, 0, 8, 128, 16, 4, None, None], "ppippiiiilpp"),
    "pa_decode_q8": ([16, 16, A, 16, 1, 16, 0, 16, 8, 128, 1, 16, 4, 0.0, 0, 256, 1 << 30, None,
                      None], "ppppipiiiiiilfipzpp"),
    "pa_rotary_store": (HEAD + [16, 16] + TAIL, "ppppllll" "iplpppp" "iiiiilpp"),
    "pa_rotary_store_q8": (HEAD + [A] + TAIL, "ppppllll" "iplppp" "iiiiilpp"),
}


@pytest.fixture(scope="module")
def calls():
    lib_build.build()
    return pk._calls()


@pytest.mark.parametrize("name", CALLS)
def test_arguments_keep_their_kind(calls, name):
    args, types = CALLS[name]
    fn = getattr(calls, name)
    assert len(args) == len(types) and fn(*args) == 0
    for i, t in enumerate(types):
        def call(x):
            return fn(*args[:i], x, *args[i + 1:])

        if t == "f":
            for x in ("x", None):
                with pytest.raises(TypeError):
                    call(x)
            assert call(1) == 0
            continue
        for x in (1.0, 0.0, "x", *(() if t == "p" else (None,))):
            with pytest.raises(TypeError):
                call(x)
        for x in {"i": (1 << 31, -(1 << 31) - 1, 1 << 32, 1 << 70), "l": (1 << 63, -(1 << 63) - 1),
                  "p": (-1, 1 << 64), "z": (-1, 1 << 64)}[t]:
            with pytest.raises(OverflowError):
                call(x)


@pytest.mark.parametrize("grid", [1 << 31, 1 << 32, -(1 << 40)])
def test_a_grid_is_not_cut_to_32_bits(grid):
    cache = pk.Q8Cache(2, 16, 8, 128, torch.int8, device="cpu")
    q, i = torch.zeros(2, 16, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(pk.PagedAttentionError, match="grid_ctas"):
        pk.pa_decode_q8(q, q, cache, i[:, None], i, grid_ctas=grid)


def build_module_under(monkeypatch, **config):
    """build.py as another interpreter would import it."""
    get = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: config.get(name, get(name)))
    spec = importlib.util.spec_from_file_location("another_build", lib_build.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_a_module_of_another_interpreter_is_not_taken(calls, monkeypatch):
    assert calls.__spec__.origin == lib_build.CALL_PATH and lib_build.up_to_date()
    other = build_module_under(monkeypatch, EXT_SUFFIX=".cpython-399-elsewhere.so")
    assert other.LIB_PATH == lib_build.LIB_PATH
    assert other.CALL_PATH != lib_build.CALL_PATH and not other.up_to_date()


def test_only_what_is_stale_is_built(calls, monkeypatch):
    made = []
    monkeypatch.setattr(lib_build, "build_call", lambda: made.append("module"))
    monkeypatch.setattr(lib_build, "_build_to", lambda path, *a: made.append(path))
    assert lib_build.build() == lib_build.LIB_PATH and made == []
    monkeypatch.setattr(lib_build, "CALL_PATH", lib_build.CALL_PATH + ".missing")
    assert lib_build.build() == lib_build.LIB_PATH and made == ["module"]
    assert lib_build.build(force=True) == lib_build.LIB_PATH
    assert sorted(made[1:]) == sorted(["module", lib_build.LIB_PATH])


def test_the_library_is_built_without_python_headers(calls, monkeypatch, tmp_path):
    """Only the module needs them, and the calls go through ctypes without it."""
    made = []
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(lib_build, "CALL_PATH", str(tmp_path / "_pa_call.so"))
    monkeypatch.setattr(lib_build, "_build_to", lambda path, *a: made.append(path))
    assert lib_build.up_to_date() and lib_build.build() == lib_build.LIB_PATH and not made
    assert lib_build.build(force=True) == lib_build.LIB_PATH and made == [lib_build.LIB_PATH]
    monkeypatch.setattr(pk, "_call_module", None)
    other = pk._calls()
    assert other is not calls
    for name, (args, types) in CALLS.items():
        fn = getattr(other, name)
        assert fn(*args) == 0
        # the module's statuses, with one argument at a time refused (nothing is ever to do)
        for i, t in enumerate(types):
            if t in "ilp":
                bad = [*args[:i], None if t == "p" else -1, *args[i + 1:]]
                assert fn(*bad) == getattr(calls, name)(*bad), (name, i)


def test_a_compiler_error_is_not_passed_over(monkeypatch, tmp_path):
    monkeypatch.setattr(lib_build, "CALL_SRC", str(tmp_path / "absent.c"))
    monkeypatch.setattr(lib_build, "CALL_PATH", str(tmp_path / "_pa_call.so"))
    with pytest.raises(RuntimeError, match="absent.c"):
        lib_build.build_call()


def test_an_interpreter_without_a_suffix(monkeypatch):
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: None)
    spec = importlib.util.spec_from_file_location("another_build", lib_build.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.CALL_PATH.endswith("_pa_call.so")
