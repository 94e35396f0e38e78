from .build import build, build_binding

if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_binding(force=True, verbose=True))
