"""The package where the compiled marshalling is not there: the optimizer needs
none of it, and the training operators say what is missing."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "zero_sharded_optimizer_step_gb300"


@pytest.fixture
def builder():
    import __graft_entry__
    zbuild = __graft_entry__._library_builder()
    zbuild.build()
    return zbuild


@pytest.fixture
def tree(tmp_path, builder):
    """The package without the marshalling module."""
    to = tmp_path / PACKAGE
    to.mkdir()
    for name in os.listdir(os.path.join(ROOT, PACKAGE)):
        if name.endswith(".py"):
            shutil.copy(os.path.join(ROOT, PACKAGE, name), str(to / name))
    os.symlink(builder.LIB, str(to / "libzero.so"))
    return tmp_path


def python(tree, code):
    env = dict(os.environ, PYTHONPATH=str(tree))
    return subprocess.run([sys.executable, "-c", code], cwd=str(tree), env=env, text=True,
                          capture_output=True, timeout=300)


def test_the_optimizer_needs_no_marshalling_module(tree):
    r = python(tree, "import %s as z\n"
                     "from %s import ZeroAdam, ShardedZeroAdam, Mx4Linear\n"
                     "assert z.zero_shard_size(10, 4) == 3\n"
                     "assert z.zero_mx4_bytes(128, 256) == 17408\n" % (PACKAGE, PACKAGE))
    assert r.returncode == 0, r.stderr


def test_the_operators_say_what_is_missing(tree):
    r = python(tree, "import %s as z\n"
                     "for call, n in [(z.zero_embed, 12), (z.zero_embed_grad, 16),\n"
                     "                (z.zero_dropout, 8), (z.zero_mx4_quantize, 6),\n"
                     "                (z.zero_mx4_dequantize, 6), (z.zero_mx4_matmul, 10)]:\n"
                     "    try:\n"
                     "        call(*[0] * n, stream=0)\n"
                     "    except ImportError as e:\n"
                     "        assert '_calls' in str(e) and 'build' in str(e), e\n"
                     "    else:\n"
                     "        raise SystemExit('%%s did not raise' %% call.__name__)\n" % PACKAGE)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_module_built_for_another_python_is_not_loaded(tree, builder):
    assert os.path.basename(builder.CALLS) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    other = builder.CALLS.replace(sysconfig.get_config_var("SOABI"), "cpython-399-other")
    assert other != builder.CALLS
    shutil.copy(builder.CALLS, str(tree / PACKAGE / os.path.basename(other)))
    r = python(tree, "import %s as z\n"
                     "try:\n"
                     "    z.zero_dropout(None, None, None, 0, 0, 0.5, 1, 2, 0, 0)\n"
                     "except ImportError:\n"
                     "    print('not loaded')\n" % PACKAGE)
    assert r.returncode == 0 and "not loaded" in r.stdout, r.stdout + r.stderr


def test_building_without_python_headers_still_builds_the_library(builder, tmp_path, monkeypatch,
                                                                 capsys):
    monkeypatch.setattr(builder, "CALLS", str(tmp_path / "calls.so"))
    monkeypatch.setattr(builder.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert builder.build() == builder.LIB and os.path.exists(builder.LIB)
    assert not os.path.exists(str(tmp_path / "calls.so"))
    assert "Python.h" in capsys.readouterr().err
